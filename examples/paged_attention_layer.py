"""One attention layer of a serving loop with everything in 4 bits: projections by gai4_qmv / gai4_qmm_t, keys and values
in a paged cache that the device itself keeps the books of.

Three requests of different lengths are read in, then continue one token a step; one ends on the way and another takes
its pages. Each step is plan -> projections -> append -> attention -> output projection, without the host reading a
length. Run it from the repository's root (a GB300 and the built library are needed):

    python examples/paged_attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_affine_int4_gb300 as g4  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, HEAD, GROUP, PAGE = 1024, 8, 2, 128, 64, 32
T = torch.bfloat16


class Layer:
    """Weights, cache and bookkeeping of one layer for up to `batch` requests of `max_len` tokens, `pages` in the pool."""

    def __init__(self, batch, max_len, pages, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def packed(n, k):
            return g4.gai4_quantize(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5, 4, GROUP, T)

        self.w_qkv = packed((Q_HEADS + 2 * KV_HEADS) * HEAD, HIDDEN)
        self.w_out = packed(HIDDEN, Q_HEADS * HEAD)
        self.k_cache = g4.gai4_kv_cache(pages, KV_HEADS, PAGE, HEAD, GROUP, T)
        self.v_cache = g4.gai4_kv_cache(pages, KV_HEADS, PAGE, HEAD, GROUP, T)
        self.table = torch.full((batch, -(-max_len // PAGE)), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.workspace = torch.empty(g4.gai4_kv_attention_workspace_bytes(Q_HEADS, KV_HEADS, HEAD, T), dtype=torch.uint8,
                                     device="cuda")

    def _project(self, w, x):
        return g4.gai4_qmm_t(*w, x, group_size=GROUP) if x.shape[0] > 1 else g4.gai4_qmv(*w, x[0], group_size=GROUP)[None]

    def step(self, x, q_lens, max_q_len):
        """x [tokens, HIDDEN]: the new tokens' activations, request after request, q_lens [batch] of them each (-1: the
        request has finished). Returns their outputs and the plan."""
        plan = g4.gai4_kv_plan(self.lens, q_lens, self.table, self.free, self.free_count, PAGE, x.shape[0])
        qkv = self._project(self.w_qkv, x).view(x.shape[0], Q_HEADS + 2 * KV_HEADS, HEAD)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)      # strided views: no copies
        # (for rotary positions, gai4_rope takes plan.positions here: fp8_decoder_layer.py)
        g4.gai4_kv_append(k, v, plan.slots, self.k_cache, self.v_cache, group_size=GROUP)
        o = g4.gai4_kv_attention(q, self.k_cache, self.v_cache, self.table, plan.kv_lens, plan.cu_q, group_size=GROUP,
                                 max_q_len=max_q_len, workspace=self.workspace)
        self.lens, self.free_count = plan.kv_lens, plan.free_count
        return self._project(self.w_out, o.view(x.shape[0], Q_HEADS * HEAD)), plan


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
