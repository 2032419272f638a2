"""A whole decoder layer of a serving loop: 8-bit floating-point products, rotary positions, and the paged 4-bit cache.

Each step is plan -> norm -> query/key/value product -> rotary positions (of plan.positions, in place) -> append ->
attention -> quantization -> output product -> norm with the residual -> gate and up product -> down product, without
the host reading a length. Activations enter every product as e4m3 with a scale for each 128; the norms write them that
way. Run it from the repository's root (a GB300 and the built library are needed):

    python examples/fp8_decoder_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_affine_int4_gb300 as g4  # noqa: E402

HIDDEN, INNER, Q_HEADS, KV_HEADS, HEAD, GROUP, PAGE = 1024, 2816, 8, 2, 128, 64, 32
T = torch.bfloat16


class Layer:
    """Weights, cache and bookkeeping of one layer for up to `batch` requests of `max_len` tokens, `pages` in the pool."""

    def __init__(self, batch, max_len, pages, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def packed(n, k):
            return g4.gai4_quantize_fp8(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)

        self.w_qkv = packed((Q_HEADS + 2 * KV_HEADS) * HEAD, HIDDEN)
        self.w_out = packed(HIDDEN, Q_HEADS * HEAD)
        self.w_gate_up = packed(2 * INNER, HIDDEN)
        self.w_down = packed(HIDDEN, INNER)
        self.gain1, self.gain2 = ((1 + 0.1 * torch.randn(HIDDEN, generator=g, device="cuda")).to(T) for _ in range(2))
        # contexts four times as long as the 8192 positions that the base is made for
        self.inv_freq, self.mscale = g4.gai4_rope_inv_freq(HEAD, 10000.0, scaling="yarn", factor=4.0, original_len=8192)
        self.k_cache = g4.gai4_kv_cache(pages, KV_HEADS, PAGE, HEAD, GROUP, T)
        self.v_cache = g4.gai4_kv_cache(pages, KV_HEADS, PAGE, HEAD, GROUP, T)
        self.table = torch.full((batch, -(-max_len // PAGE)), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device="cuda")

    def step(self, x, q_lens, max_q_len):
        """x [tokens, HIDDEN]: the new tokens' activations, request after request, q_lens [batch] of them each (-1: the
        request has finished). Returns their outputs and the plan."""
        n = x.shape[0]
        plan = g4.gai4_kv_plan(self.lens, q_lens, self.table, self.free, self.free_count, PAGE, n)
        h = g4.gai4_rms_norm(x, self.gain1, fp8=True)
        qkv = g4.gai4_fp8_mm_t(*self.w_qkv, h.codes, h.scales, dtype=T).view(n, Q_HEADS + 2 * KV_HEADS, HEAD)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)      # strided views: no copies
        g4.gai4_rope(q, k, plan.positions, self.inv_freq, mscale=self.mscale, q_out=q, k_out=k)
        g4.gai4_kv_append(k, v, plan.slots, self.k_cache, self.v_cache, group_size=GROUP)
        o = g4.gai4_kv_attention(q, self.k_cache, self.v_cache, self.table, plan.kv_lens, plan.cu_q, group_size=GROUP,
                                 max_q_len=max_q_len)
        a = g4.gai4_fp8_mm_t(*self.w_out, *g4.gai4_quantize_x_fp8(o.view(n, Q_HEADS * HEAD)), dtype=T)
        h = g4.gai4_rms_norm(a, self.gain2, residual=x, fp8=True)
        gate, up = g4.gai4_fp8_mm_t(*self.w_gate_up, h.codes, h.scales, dtype=T).chunk(2, 1)
        m = torch.nn.functional.silu(gate) * up
        y = g4.gai4_fp8_mm_t(*self.w_down, *g4.gai4_quantize_x_fp8(m), dtype=T) + h.residual
        self.lens, self.free_count = plan.kv_lens, plan.free_count
        return y, plan


def main():
    torch.manual_seed(1)
    layer = Layer(batch=3, max_len=512, pages=24)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    steps = [((300, 45, 120), 300)] + [((1, 1, 1), 1)] * 4 + [((1, -1, 1), 1), ((1, 200, 1), 200)] + [((1, 1, 1), 1)] * 3
    for lens, longest in steps:
        x = torch.randn(sum(max(n, 0) for n in lens), HIDDEN, device="cuda").to(T)
        y, plan = layer.step(x, ints(*lens), longest)
        print(f"new {str(lens):18} cached {str(plan.kv_lens.tolist()):16} free pages {int(plan.free_count):3} "
              f"output rms {float(y.float().square().mean().sqrt()):.4f}")
        assert plan.info.tolist() == [0, 0, 0, 0] and bool(y.isfinite().all())
    assert g4.gai4_last_device_status() == g4.GAI4_OK
    return layer


if __name__ == "__main__":
    main()
