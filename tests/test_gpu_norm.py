"""ss_rmsnorm_act on the GPU against the oracle, bit for bit: the mean is summed in float64 on both sides, so whatever the
order of the sums, the root rounds to the same float32, and every later step is one float32 rounding."""
import numpy as np
import pytest
import torch

import oracle
from helpers import dev_bf16, dev_f32, have_gpu, host
from oracle.norm import codes, rmsnorm

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ss():
    import structured_sparse_quantized_amd as m
    return m


def _rows(rng, M, K, bf16, ld=None, size=1.0):
    """Values of the type, and a device matrix whose rows start on 16 bytes."""
    per = 8 if bf16 else 4
    ld = ld or (K + per - 1) // per * per
    x = (size * rng.standard_normal((M, ld)) * np.exp(rng.standard_normal(ld))).astype(np.float32)
    if bf16:
        b = oracle.f32_to_bf16_bits_rne(x)
        return oracle.bf16_bits_to_f32(b)[:, :K], dev_bf16(b)[:, :K]
    return x[:, :K], dev_f32(x)[:, :K]


def _weights(rng, K, kind):
    w = (0.1 + rng.random(K)).astype(np.float32)
    if kind == "bf16":
        b = oracle.f32_to_bf16_bits_rne(w)
        return oracle.bf16_bits_to_f32(b), dev_bf16(b)
    return (w, dev_f32(w)) if kind == "f32" else (None, None)


def _check(got, exp, y, n):
    z, r = exp
    out, sx, total = got
    if y == "bf16":
        assert sx is None and np.array_equal(host(out), oracle.f32_to_bf16_bits_rne(z))
    else:
        c, s = codes(z, n, y)
        assert np.array_equal(host(sx), s)
        assert np.array_equal(host(out), c)
    if total is not None:
        assert np.array_equal(total.float().cpu().numpy(), r)


SIZES = [1, 3, 7, 8, 9, 64, 100, 511, 512, 513, 1501, 2048, 3584, 4096, 5000, 8200, 16384, 20001, 32768, 32769, 40000]


@pytest.mark.parametrize("K", SIZES)
@pytest.mark.parametrize("x,w,res", [("bf16", "bf16", True), ("bf16", "f32", False), ("f32", "f32", True), ("f32", None, False)])
@pytest.mark.parametrize("y", ["bf16", "i8", "fp8"])
def test_sizes_and_types(ss, K, x, w, res, y):
    rng = np.random.default_rng(K)
    M = 3 if K > 5000 else 17
    a, ta = _rows(rng, M, K, x == "bf16")
    b, tb = _rows(rng, M, K, x == "bf16") if res else (None, None)
    wv, tw = _weights(rng, K, w)
    _check(ss.rmsnorm_act(ta, tw, 1e-5, residual=tb, y_dtype=y), rmsnorm(a, wv, 1e-5, b, x == "bf16"), y, 2)


@pytest.mark.parametrize("n", range(2, 9))
@pytest.mark.parametrize("K", [5, 8, 120, 1000, 3584, 4102, 17000, 33001])
@pytest.mark.parametrize("x,y", [("bf16", "i8"), ("f32", "fp8")])
def test_every_lift(ss, n, K, x, y):
    rng = np.random.default_rng(K + n)
    M = 2 if K > 10000 else 5
    a, ta = _rows(rng, M, K, x == "bf16")
    wv, tw = _weights(rng, K, x)
    _check(ss.rmsnorm_act(ta, tw, 1e-6, n=n, y_dtype=y), rmsnorm(a, wv, 1e-6, None, x == "bf16"), y, n)


def test_is_a_step_of_the_quantiser_on_the_normalised_rows(ss):
    """inv is rounded once there and twice here: the codes are equal but at borders, the scales equal."""
    rng = np.random.default_rng(5)
    a, ta = _rows(rng, 40, 1504, True)
    wv, tw = _weights(rng, 1504, "bf16")
    z, _ = rmsnorm(a, wv, 1e-5)
    for n in (2, 3, 4):
        for q in ("i8", "fp8"):
            y, sx, _ = ss.rmsnorm_act(ta, tw, 1e-5, n=n, y_dtype=q)
            y2, sx2 = ss.quant_lift_act(dev_f32(z), n, q)
            d = y.float() - y2.float()
            assert torch.equal(sx, sx2) and (d.abs() <= (1 if q == "i8" else 2.0 ** -3 * y2.float().abs() + 2.0 ** -9)).all()
            assert (d != 0).float().mean() < 1e-3  # borders are 2^-22 of a step wide


@pytest.mark.parametrize("y", ["i8", "fp8"])
def test_equals_elementwise_tensor_operations(ss, y):
    rng = np.random.default_rng(8)
    _, x = _rows(rng, 300, 4096, True)
    _, res = _rows(rng, 300, 4096, True)
    _, w = _weights(rng, 4096, "bf16")
    r = (x.float() + res.float()).to(torch.bfloat16)
    z = r.float() * (1 / torch.sqrt(r.double().square().mean(1, keepdim=True) + 1e-5)).float() * w.float()
    top = 127.0 if y == "i8" else 448.0
    t = (z * (top / z.abs().amax(1, keepdim=True))).clamp(-top, top)
    got = ss.rmsnorm_act(x, w, 1e-5, residual=res, y_dtype=y)
    assert torch.equal(got[2], r)
    exp = t.round().to(torch.int8) if y == "i8" else t.to(torch.float8_e4m3fn)
    assert torch.equal(got[0].float(), exp.float())


@pytest.mark.parametrize("K", [100, 4096, 40000])
@pytest.mark.parametrize("bf16", [True, False])
def test_in_place_and_given_outputs(ss, K, bf16):
    """sum over the residual or over x, rows with room behind them, whose tails stay as they are."""
    rng = np.random.default_rng(K)
    ld = (K + 31) // 8 * 8
    a, ta = _rows(rng, 9, K, bf16, ld)
    b, tb = _rows(rng, 9, K, bf16, ld)
    wv, tw = _weights(rng, K, "f32")
    exp = rmsnorm(a, wv, 1e-5, b, bf16)
    z = exp[0]
    for into in ("residual", "x"):
        x, r = ta._base.clone(), tb._base.clone()
        tail = (r if into == "residual" else x)[:, K:].clone()
        whole = torch.full((9, oracle.lifted_k_alloc(K, 2) + 16), 77, dtype=torch.int8, device="cuda")
        sx = torch.full((12,), 5.0, device="cuda")
        got = ss.rmsnorm_act(x[:, :K], tw, 1e-5, residual=r[:, :K], y_dtype="i8", sum_out=(r if into == "residual" else x)[:, :K],
                             out=whole, scale_out=sx)
        c, s = codes(z, 2, "i8")
        assert got[0].data_ptr() == whole.data_ptr() and np.array_equal(host(whole[:, : c.shape[1]]), c)
        assert (whole[:, c.shape[1] :] == 77).all() and np.array_equal(host(sx[:9]), s) and (sx[9:] == 5).all()
        kept = r if into == "residual" else x
        assert np.array_equal(kept[:, :K].float().cpu().numpy(), exp[1]) and torch.equal(kept[:, K:], tail)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 2.5])
def test_rows_of_zeros_and_extreme_sizes(ss, eps):
    rng = np.random.default_rng(3)
    a = rng.standard_normal((6, 640)).astype(np.float32)
    a[1] = 0
    a[2] *= 1e-18
    a[3] *= 1e18  # squares beyond float32
    a[4, 1:] = 0
    wv, tw = _weights(rng, 640, "f32")
    for y in ("bf16", "i8", "fp8"):
        _check(ss.rmsnorm_act(dev_f32(a), tw, eps, y_dtype=y), rmsnorm(a, wv, eps, None, False), y, 2)


def test_many_short_rows(ss):
    """Norms of single heads: 70001 rows of 128."""
    rng = np.random.default_rng(4)
    a, ta = _rows(rng, 70001, 128, True)
    wv, tw = _weights(rng, 128, "bf16")
    _check(ss.rmsnorm_act(ta, tw, 1e-6), rmsnorm(a, wv, 1e-6), "bf16", 2)


def test_rows_far_apart(ss):
    """Rows beyond 2^31 elements of their matrices."""
    ld = 1 << 30
    x = torch.zeros((3, ld), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros((3, ld), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(6)
    a, ta = _rows(rng, 3, 520, True)
    b, tb = _rows(rng, 3, 520, True)
    x[:, :520], r[:, :520] = ta, tb
    out = torch.empty((3, ld * 2), dtype=torch.int8, device="cuda")
    got = ss.rmsnorm_act(x[:, :520], None, 1e-6, residual=r[:, :520], y_dtype="i8", sum_out=r[:, :520], out=out)
    _check((out[:, :768], got[1], got[2]), rmsnorm(a, None, 1e-6, b), "i8", 2)


def test_streams_and_graphs(ss):
    rng = np.random.default_rng(7)
    a, ta = _rows(rng, 33, 2000, True)
    b, tb = _rows(rng, 33, 2000, True)
    wv, tw = _weights(rng, 2000, "bf16")
    exp = rmsnorm(a, wv, 1e-6, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _check(ss.rmsnorm_act(ta, tw, residual=tb, n=4, y_dtype="i8"), exp, "i8", 4)
    x = ta.clone()
    graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph):
        got = ss.rmsnorm_act(x, tw, residual=tb, n=4, y_dtype="i8")
    for k in range(3):
        c, tc = _rows(rng, 33, 2000, True)
        x.copy_(tc)
        graph.replay()
        torch.cuda.synchronize()
        _check(got, rmsnorm(c, wv, 1e-6, b), "i8", 4)
