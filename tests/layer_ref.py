"""64-bit references and error bounds of the operators around the attention (rotary positions, norm, e4m3 quantization
and product). U(T) is half a step of T relative to a value (finfo.eps / 2); u = 2^-24 is binary32's."""
import torch

u = 2.0 ** -24
U = {torch.float32: u, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
E4M3 = torch.float8_e4m3fn


def within(got, ref, bound, what=""):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = ((got - ref).abs() / bound).nan_to_num(1e30).where(bad, torch.zeros_like(ref)).argmax()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {got.flatten()[i]} for "
                             f"{ref.flatten()[i]}, bound {bound.expand_as(ref).flatten()[i]}")


def rope64(x, positions, inv_freq, mscale, interleaved):
    """(values, bound). A kernel's argument of sine and cosine, in half turns below 1, is rounded once (pi u of an
    angle), their results by at most an ulp each (2 u), mscale's product, two products and their sum by u each: below
    8 u (|a| + |b|) mscale with a spare u for the turn's 64-bit fraction; then the output."""
    half = inv_freq.shape[0]
    t = positions.double()[:, None] * inv_freq.double()
    c, s = torch.cos(t)[:, None] * mscale, torch.sin(t)[:, None] * mscale
    y = x.double().clone()
    r = x.double()[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    p, q = a * c - b * s, b * c + a * s
    m = 8 * u * abs(mscale) * (a.abs() + b.abs())
    bound = torch.zeros_like(y)
    for to, v in ((y, (p, q)), (bound, (m, m))):
        to[..., :2 * half] = torch.stack(v, -1).flatten(-2) if interleaved else torch.cat(v, -1)
    turned = torch.zeros_like(y)
    turned[..., :2 * half] = 1
    return y, bound * (1 + U[x.dtype]) + turned * (U[x.dtype] * y.abs() + TINY[x.dtype])


def norm64(x, gain, eps, residual, a_warp_a_row=False):
    """(h, y, relative bound of y before its last rounding). The sum of squares goes through at most 8 + 4 + 10 additions
    (8 + cols / 8192 + 10 for long rows) and counts half in y; x + residual, the mean, eps, the root and two products
    round once each, h in the sum and in y. A warp that takes a row in steps of 256 adds 8 squares a lane, a step at a
    time, and 32 lanes: 8 + cols / 256 + 5."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    if gain is not None:
        y = y * gain.double()
    additions = 14 + h.shape[1] / 256 if a_warp_a_row else 22 + h.shape[1] / 8192
    return h, y, u * additions / 2 + 8 * u


def quantize_ref(x, block_rows):
    """e4m3 codes and scales by the rule, bit for bit: x [R, C] with blocks of block_rows x 128."""
    R, C = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -C % 128, 0, -R % block_rows))
    b = p.unflatten(0, (-1, block_rows)).unflatten(2, (-1, 128))
    a = b.abs().amax((1, 3), keepdim=True).clamp(min=2.0 ** -100)
    q = (b.double() * 448 / a.double()).float()
    q = q.flatten(2).flatten(0, 1)[:R, :C]
    return q.to(E4M3), (a / torch.full_like(a, 448.0))[:, 0, :, 0]


def values(codes, scales, block_rows):
    R, C = codes.shape
    s = scales.double().repeat_interleave(128, 1)[:, :C]
    return codes.double() * (s if block_rows == 1 else s.repeat_interleave(block_rows, 0)[:R])


def mm64(wc, ws, xc, xs, dtype):
    """(values, bound). Of the sum of absolute products: the tensor core's sums of a block, four steps of 32 products and
    the sum so far, each aligned to the largest and cut off at no less than 24 bits, 132 u; the product of two scales
    and the product with it, 2 u; an addition a block; then the output."""
    w, x = values(wc, ws, 128), values(xc, xs, 1)
    y, m = x @ w.t(), x.abs() @ w.abs().t()
    blocks = -(-wc.shape[1] // 128)
    return y, m * u * (134 + blocks) + U[dtype] * y.abs() + TINY[dtype]
