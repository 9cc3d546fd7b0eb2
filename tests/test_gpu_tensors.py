"""The binding's quick look at a call's tensors (`_tensors`) against its slow one: the
same pointers where a tensor is as it must be, and the slow one's error where it is not
(needs an MI355X; what the module says of CPU tensors is in tests/test_tensors.py).
"""

import pytest

from bit_quantized_linear_amd import binding as b
from tests import gpu_harness as H
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def quick():
    calls = b._quick()
    assert len(calls) == 7, "built with the library"
    return calls


def test_pointers_are_those_of_the_tensors():
    t = H.torch()
    pointers, _, e4m3, bf16, f32, i32, f64 = quick()
    dev = t.cuda.current_device()
    for kind, types in ((e4m3, (t.float8_e4m3fn, t.uint8, t.int8)), (bf16, (t.bfloat16, t.int16, t.uint16)), (f32, (t.float32,)),
                        (i32, (t.int32, t.uint32)), (f64, (t.float64,))):
        every = [t.empty((6, 8), dtype=d, device="cuda") for d in
                 (t.float8_e4m3fn, t.uint8, t.int8, t.bfloat16, t.int16, t.uint16, t.float32, t.int32, t.uint32, t.float64,
                  t.float16, t.float8_e5m2, t.float8_e4m3fnuz, t.int64, t.bool)]
        for x in every:
            got = pointers(dev, x[2:], kind, (4, 8), None, kind, 5)
            assert got == ((x[2:].data_ptr(), None) if x.dtype in types else None), (x.dtype, types)


def test_what_it_refuses():
    t = H.torch()
    pointers, heads, _, bf16, _, _, _ = quick()
    dev = t.cuda.current_device()
    x = t.zeros((6, 8), dtype=t.bfloat16, device="cuda")
    assert pointers(dev, x, bf16, 96) == (x.data_ptr(),) == pointers(dev, x, bf16, (6, 8)) == pointers(dev, x, b._ANY_KIND, 0)
    for tensor, need in ((x, 97), (x, (8, 6)), (x, (6, 8, 1)), (x, (48,)), (x, "96"), (x, (6, "8")), (x.t(), 96), (x[:, :4], 0),
                         (x.cpu(), 96), (x.half(), 96), (t.nn.Parameter(x), 96), (x.to_sparse(), 0), (3, 0), ("x", 0)):
        assert pointers(dev, tensor, bf16, need) is None
    assert pointers(dev + 1, x, bf16, 0) is None
    q = t.zeros((5, 6, 64), dtype=t.bfloat16, device="cuda")
    assert heads(dev, bf16, q[:, 2:4]) == (q[:, 2:4].data_ptr(), 384, 5, 2, 64)
    for bad in (q[:, ::2], q.transpose(0, 1), q[..., ::2], q[0], q.half(), q.cpu(), q[:1].expand(5, 6, 64), None):
        assert heads(dev, bf16, bad) is None
    with pytest.raises(TypeError):
        pointers(dev, x, bf16)
    with pytest.raises(TypeError):
        heads(dev, bf16)


@pytest.mark.parametrize("shape,cut", [((5, 6, 64), (slice(None), slice(1, 3))), ((1, 6, 64), (slice(None), slice(1, 3))),
                                       ((0, 6, 64), (slice(None),)), ((4, 1, 80), (slice(None),)), ((3, 0, 64), (slice(None),)),
                                       ((1, 5, 8), (slice(None),)), ((7, 2, 64), (slice(None, None, 2),))])
def test_heads_as_the_slow_look(shape, cut, monkeypatch):
    t = H.torch()
    x = t.zeros(shape, dtype=t.bfloat16, device="cuda")[cut]
    fast = b._dev_heads(x, "X", t.cuda.current_device())
    monkeypatch.setattr(b, "_quick_calls", ())
    assert fast == b._dev_heads(x, "X", t.cuda.current_device())


def test_errors_are_the_slow_looks():
    t = H.torch()
    x = t.zeros((4, 128), dtype=t.bfloat16, device="cuda")
    qx, sx = t.zeros((4, 128), dtype=t.uint8, device="cuda"), t.zeros((1, 4), device="cuda")
    w = t.ones(128, dtype=t.bfloat16, device="cuda")
    b.svdq_fp8_norm_quantize(x, None, w, 1e-6, None, None, qx, sx)
    b.svdq_fp8_norm_quantize(x, None, t.nn.Parameter(w), 1e-6, None, None, qx, sx.flatten())  # as the slow look takes them
    for change, error in (({"x": x.half()}, TypeError), ({"w": w.cpu()}, TypeError), ({"qx": qx[:2]}, ValueError),
                          ({"sx": sx.t().contiguous()}, ValueError), ({"x": x.t()}, TypeError), ({"w": w[:64]}, ValueError)):
        a = {"x": x, "w": w, "qx": qx, "sx": sx, **change}
        with pytest.raises(error):
            b.svdq_fp8_norm_quantize(a["x"], None, a["w"], 1e-6, None, None, a["qx"], a["sx"])
    kc, vc = (t.zeros((3, 2) + s, dtype=t.uint8, device="cuda") for s in ((64, 128), (128, 64)))
    s = t.ones((3, 2), device="cuda")
    k = t.zeros((2, 2, 128), dtype=t.bfloat16, device="cuda")
    starts, lengths, table = (t.tensor(v, dtype=t.int32, device="cuda") for v in ([0, 2], [2], [[1]]))
    good = dict(K=k, V=k, starts=starts, lengths=lengths, table=table, kc=kc, ks=s, vc=vc, vs=s)
    b.svdq_kv8_append(**good)
    for change, error in (({"kc": vc}, ValueError), ({"ks": s.t()}, ValueError), ({"starts": starts[:1]}, ValueError),
                          ({"table": table.long()}, TypeError), ({"lengths": lengths.cpu()}, TypeError),
                          ({"K": k[:, :1]}, ValueError), ({"vs": s.double()}, TypeError)):
        with pytest.raises(error):
            b.svdq_kv8_append(**{**good, **change})
    o = t.zeros((2, 2, 128), dtype=t.bfloat16, device="cuda")
    call = lambda **c: b.svdq_kv8_attention(k, kc, s, vc, s, starts, lengths, table, 0.1, c.pop("O", o), **c)  # noqa: E731
    call(lse=t.zeros((2, 2), device="cuda"), workspace=t.zeros(3, dtype=t.float64, device="cuda"))
    for change, error in (({"O": o[:1]}, ValueError), ({"lse": t.zeros((2, 3), device="cuda")}, ValueError),
                          ({"workspace": t.zeros(8)}, TypeError), ({"O": o.float()}, TypeError)):
        with pytest.raises(error):
            call(**change)
