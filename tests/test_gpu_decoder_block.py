"""The attention half of a decoder block as a program runs it, a prompt and then
decoded tokens: norm -> block-scaled FP8 projection -> rotary positions in place ->
append -> attention -> FP8 projection -> norm with the residual -> experts. Each step
is held against the oracle's on what the library's last step wrote (needs an MI355X).

Tolerances as in the steps' own tests (test_gpu_norm_rope.py, test_gpu_kv8.py,
test_gpu_fp8.py); a product of the norm's codes is held against the matrix core's own
sums of them (oracle/fp8.py, F5).
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl
from oracle import decoder as od
from oracle import fp8 as of8
from tests import gpu_harness as H
from tests.test_gpu_fp8 import check as check_linear
from tests.test_gpu_kv8 import check as check_attention
from tests.test_gpu_norm_rope import _gpu, norm_check, rope_check, values  # noqa: F401

pytestmark = pytest.mark.gpu

K, HQ, HK, D, E, I = 512, 6, 2, 64, 6, 64  # noqa: E741
SECTIONS, EPS, THETA = (16, 8, 8), 1e-5, 10000.0
N = (HQ + 2 * HK) * D


class Block:
    def __init__(self, sequences, pages):
        t = self.t = H.torch()
        rng = np.random.default_rng(1)
        bf = lambda seed, shape, std: wl.random_bf16(seed, shape, std)  # noqa: E731
        self.w1, self.w2 = (bf(s, (K,), 0.2) for s in (2, 3))
        self.qkv = of8.prepare_weights(bf(4, (K, N), 0.06)["values"])
        self.out = of8.prepare_weights(bf(5, (HQ * D, K), 0.05)["values"])
        self.bias = bf(6, (N,), 0.05)
        self.wr = bf(7, (E, K), 0.2)
        stack = lambda seed, n, shape: [np.stack(z) for z in zip(*(of8.prepare_weights(  # noqa: E731
            bf(seed + i, shape, 0.05)["values"]) for i in range(n)))]
        q13, s13 = stack(20, 2 * E, (K, I))
        self.w13 = q13.reshape(E, 2, I, K), s13.reshape(E, 2, *s13.shape[1:])
        self.w2e = stack(60, E, (I, K))
        self.freqs = np.concatenate([THETA ** (-np.arange(n) / n) for n in SECTIONS])
        rand = lambda *s: rng.integers(0, 0x7E, s).astype(np.uint8)  # noqa: E731
        self.cache = od.Cache(rand(pages, HK, 64, D), np.ones((pages, HK), np.float32), rand(pages, HK, D, 64),
                              np.ones((pages, HK), np.float32))
        self.dev = {n: H.dev(getattr(self.cache, n)) for n in ("kc", "ks", "vc", "vs")}
        self.order = rng.permutation(pages).tolist()
        self.table = np.full((sequences, pages), -1, np.int32)
        self.lengths = [0] * sequences
        self.d = {n: H.dev(a) for n, a in (("w1", self.w1["bits"]), ("w2", self.w2["bits"]), ("q1", self.qkv[0]),
                                           ("s1", self.qkv[1]), ("q2", self.out[0]), ("s2", self.out[1]),
                                           ("bias", self.bias["bits"]), ("wr", self.wr["bits"]), ("q13", self.w13[0]),
                                           ("s13", self.w13[1]), ("q2e", self.w2e[0]), ("s2e", self.w2e[1]),
                                           ("freqs", self.freqs))}

    def place(self, new):
        for s, n in enumerate(new):
            self.lengths[s] += n
            while np.count_nonzero(self.table[s] >= 0) * 64 < self.lengths[s]:
                self.table[s, np.count_nonzero(self.table[s] >= 0)] = self.order.pop()
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(self.lengths, new)])
        return starts, np.stack([pos // 35, pos // 7 % 5, pos % 7], 1).astype(np.int32)  # frames of 5 x 7

    def step(self, x, new):
        """x: residual stream (bf16 bits) of the new tokens; the next one's tensor."""
        t, d = self.t, self.d
        T = x.shape[0]
        starts, pos = self.place(new)
        bf = lambda *s: t.empty(s, dtype=t.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: t.empty(s, device="cuda")  # noqa: E731
        u8 = lambda *s: t.empty(s, dtype=t.uint8, device="cuda")  # noqa: E731
        xd, sd, ld, td, pd = (H.dev(a) for a in (x, starts, np.asarray(self.lengths, np.int32), self.table, pos))
        xd = xd.view(t.bfloat16)
        qx, sx, qkv = u8(T, K), f32(b.fp8_blocks(K), T), bf(T, N)
        b.svdq_fp8_norm_quantize(xd, None, d["w1"], EPS, None, None, qx, sx)
        b.svdq_fp8_gemm(qx, sx, d["q1"], d["s1"], d["bias"], qkv)
        heads = qkv.view(T, HQ + 2 * HK, D)
        before = values(heads)
        b.svdq_rope(heads[:, : HQ + HK], pd, d["freqs"], SECTIONS, heads[:, : HQ + HK])
        b.svdq_kv8_append(heads[:, HQ: HQ + HK], heads[:, HQ + HK:], sd, ld, td, *self.dev.values())
        O, L = bf(T, HQ, D), f32(T, HQ)  # noqa: E741
        ws = u8(b.svdq_kv8_attention_workspace_bytes(T, len(new), self.table.shape[1], HQ, HK, D))
        b.svdq_kv8_attention(heads[:, :HQ], *self.dev.values(), sd, ld, td, D ** -0.5, O, L, ws)
        wl2, Y = u8(b.svdq_fp8_workspace_bytes(T, HQ * D)), bf(T, K)
        b.svdq_fp8_linear(O.view(T, HQ * D), d["q2"], d["s2"], None, wl2, Y)
        xn, h = xd.clone(), bf(T, K)
        b.svdq_fp8_norm_quantize(Y, xn, d["w2"], EPS, xn, h, None, None)
        t.cuda.synchronize()
        # each step on what the library's last one wrote
        xv = wl.f32_from_bf16_bits(x).astype(np.float64)
        eps = np.float64(np.float32(EPS))
        norm_check({"qx": qx, "sx": sx}, od.norm(xv, None, self.w1["values"], eps))
        codes, scales = H.host(qx), H.host(sx)
        mag = np.abs(of8.dequantize_activations(codes, scales)) @ np.abs(of8.dequantize(*self.qkv)).T
        check_linear(before.reshape(T, N), {"y": of8.forward_cut(codes, scales, *self.qkv, self.bias["values"]), "mag": mag,
                                            "peaks": 0.0}, K, "bf16")
        turned = values(heads)
        rope_check(turned[:, : HQ + HK], before[:, : HQ + HK], pos, self.freqs, SECTIONS, False)
        assert np.array_equal(turned[:, HQ + HK:], before[:, HQ + HK:])
        self.cache.append(turned[:, HQ: HQ + HK], turned[:, HQ + HK:], starts, self.lengths, self.table)
        for n, a in self.dev.items():
            assert np.array_equal(H.host(a), getattr(self.cache, n)), n
        att = od.attention(turned[:, :HQ], self.cache, starts, self.lengths, self.table, np.float64(np.float32(D ** -0.5)))
        check_attention((values(O), H.host(L).astype(np.float64)), att, self.lengths, D)
        ref = of8.forward(values(O).reshape(T, HQ * D), *self.out, None)
        check_linear(values(Y), ref, HQ * D, "bf16")
        norm_check({"sum": xn, "Y": h}, od.norm(values(Y), xv, self.w2["values"], eps))
        if T <= b.FP8_MOE_MAX_TOKENS:  # the experts take the norm's bf16
            Ye, idx = bf(T, K), t.empty((T, 2), dtype=t.int32, device="cuda")
            wse = u8(b.svdq_fp8_moe_workspace_bytes(T, I, E, 2))
            b.svdq_fp8_moe_layer(h, d["wr"], d["q13"], d["s13"], d["q2e"], d["s2e"], Ye, idx, None, wse)
            refe = of8.moe(values(h), self.wr["values"], *self.w13, *self.w2e, 2, True)
            y = values(Ye)
            assert np.array_equal(H.host(idx), refe["idx"])
            assert np.linalg.norm(y - refe["y"]) <= 4e-3 * np.linalg.norm(refe["y"])
        return H.host(xn.view(t.int16)).view(np.uint16)


def test_a_prompt_and_decoded_tokens():
    block = Block(3, 12)
    block.step(wl.random_bf16(100, (75 + 130 + 9, K))["bits"], [75, 130, 9])
    for i in range(4):
        new = [[1, 1, 1], [1, 1, 1], [2, 1, 60], [1, 0, 1]][i]
        block.step(wl.random_bf16(101 + i, (sum(new), K))["bits"], new)


def test_layers_on_the_stream_of_the_last():
    """The residual stream of one step is the next one's input, sequences of one token."""
    block = Block(2, 6)
    x = wl.random_bf16(200, (2, K))["bits"]
    for i in range(3):
        x = block.step(x, [1, 1])
        assert np.isfinite(wl.f32_from_bf16_bits(x)).all()
