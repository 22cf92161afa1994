"""GPU tests of the fused residual addition, RMS norm and per-token quantiser.

Against the definition, in numpy:
* residual_out, and the codes where the scale is neither floored nor bounded, bit for bit (they depend on
  no sum): t = r * w, a = max |t|, inv = qmax * (1 / a), each step one binary32
  operation;
* everything against the formula in 64 bits.  With u = 2^-24 (half a binary32 step):
  - a square passes at most k/256 + 16 additions: those of its 16-byte vector (8 or 4), of its thread's
    vectors (1 up to k = 256, 2 to 512, 4 to 1024, never more than 8), 5 in the warp, 5 between warps (none up
    to k = 1024): relative error of the sum (k/256 + 16) u, halved by the square root, then the mean, eps,
    square root and reciprocal: rstd within ((k/256 + 16)/2 + 4) u;
  - scale: + 3 u (a's own rounding, z, the division); norm_out in binary32: + 2 u (t, the product);
    in bf16 half a step, 2^-8, more;
  - a code differs from qmax * t / a by at most half a unit (int8) plus five roundings of at most
    127 u; e4m3: half a step, 2^-4 relative (2^-10 among the subnormals)."""
import numpy as np
import pytest

from gpu_util import assert_bits, dev, host, need_gpu, x_dev
from oracle.oracle import Oracle
from w8a8_int8_quantized_qk_b200 import qk, synth

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module")
def O():
    need_gpu()
    return Oracle(nthreads=4)


def f32(a):
    return synth.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a


def as_type(a, bf16):
    return synth.to_bf16_bits(a) if bf16 else np.ascontiguousarray(a, np.float32)


def make(m, k, bf16, seed, residual=True):
    r = synth.streams(seed, ["x", "res", "w"])
    x = r["x"].standard_normal((m, k)).astype(np.float32)
    x[:, r["x"].choice(k, max(1, k // 100), replace=False)] *= 20.0
    res = 2.0 * r["res"].standard_normal((m, k)).astype(np.float32)
    w = 1.0 + 0.2 * r["w"].standard_normal(k).astype(np.float32)
    return as_type(x, bf16), as_type(res, bf16) if residual else None, as_type(w, bf16)


def check(O, x, res, w, eps, got, fp8=False, ub=None):
    q, scale, ro, y = got
    bf16 = x.dtype == np.uint16
    k = x.shape[1]
    r = x if res is None else as_type(f32(x) + f32(res), bf16)
    if ro is not None:
        assert_bits(host(ro), r, "residual_out")
    r32, w32, qmax = f32(r), f32(w), 448.0 if fp8 else 127.0
    t = r32 * w32
    r64, t64 = r32.astype(np.float64), r32.astype(np.float64) * w32.astype(np.float64)
    a64 = np.abs(t64).max(1)
    rstd = 1.0 / np.sqrt((r64 * r64).mean(1) + np.float64(np.float32(eps)))
    whole = np.maximum(a64 * rstd, float(np.float32(1e-12))) / qmax
    want = whole if ub is None else np.minimum(whole, np.float64(np.float32(ub)))
    tol = ((k / 256 + 16) / 2 + 4) * U
    s = host(scale).astype(np.float64)
    assert np.all(np.abs(s - want) <= want * (tol + 3 * U)), "scale"
    # codes
    free = (whole == want) & (a64 * rstd > 1.001e-12)
    codes = host(q)
    with np.errstate(all="ignore"):
        inv = np.float32(qmax) * (np.float32(1) / np.abs(t).max(1))
        v32 = t * inv[:, None]
    if fp8:
        assert_bits(codes[free], O.f32_to_e4m3(np.clip(v32[free], -448, 448).astype(np.float32)), "codes")
        val = O.e4m3_to_f32(codes).astype(np.float64)
        v = np.clip(t64 * rstd[:, None] / want[:, None], -448, 448)
        assert np.all(np.abs(val - v) <= np.abs(v) * (2.0 ** -4 + 2 * tol + 8 * U) + 2.0 ** -10), "e4m3 values"
    else:
        assert_bits(codes[free], np.rint(v32[free]).astype(np.int8), "codes")
        v = t64 * rstd[:, None] / want[:, None]
        assert np.all(np.abs(codes - v) <= 0.5 + 127 * (2 * tol + 8 * U)), "codes against 64 bits"
        assert np.all(np.abs(codes[free] - v[free]) <= 0.5 + 127 * 5 * U), "codes against 64 bits"
        assert codes.min() >= -127
    if y is not None:
        want_y = t64 * rstd[:, None]
        step = 2.0 ** -8 if bf16 else 0.0
        assert np.all(np.abs(f32(host(y)) - want_y) <= np.abs(want_y) * (step + tol + 4 * U) + 1e-40), "norm_out"


# one row to many (the forms for few and many rows), rows of one vector, rows that fill no vector count evenly,
# rows over one block's and over one cluster's registers
SHAPES = [(1, 16), (1, 4096), (2, 48), (3, 64), (5, 528), (64, 8192), (147, 1040), (297, 2064), (300, 16),
          (600, 4096), (1200, 272), (513, 8208), (2, 16400), (3, 40000), (1, 70000), (2, 140000), (1000, 16384)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
def test_norm_int8(O, m, k, bf16):
    x, res, w = make(m, k, bf16, seed=m + k)
    got = qk.add_rmsnorm_quant_per_token(x_dev(x), x_dev(w), x_dev(res), 1e-6, want_norm=True)
    check(O, x, res, w, 1e-6, got)


@pytest.mark.parametrize("vectors", [2, 32, 34, 64, 66, 128, 130, 256, 258, 512, 514, 1024, 1026, 1536, 1538, 2052])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_many_rows_of_every_width(O, vectors, bf16, residual):
    """Both sides of every choice of threads and vectors a thread, for rows enough to be walked."""
    m, k = 700, vectors * (8 if bf16 else 4) // 16 * 16 or 16
    x, res, w = make(m, k, bf16, seed=vectors, residual=residual)
    got = qk.add_rmsnorm_quant_per_token(x_dev(x), x_dev(w), x_dev(res) if residual else None, 1e-6, want_norm=True)
    check(O, x, res, w, 1e-6, got)


@pytest.mark.parametrize("m,k", SHAPES[::2])
@pytest.mark.parametrize("bf16", [True, False])
def test_norm_without_residual(O, m, k, bf16):
    x, _, w = make(m, k, bf16, seed=m * 3 + k, residual=False)
    got = qk.add_rmsnorm_quant_per_token(x_dev(x), x_dev(w), eps=1e-5)
    assert got[2] is None and got[3] is None
    check(O, x, None, w, 1e-5, got)


@pytest.mark.parametrize("m,k", SHAPES[1::2])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("ub", [None, 0.03])
def test_norm_fp8(O, m, k, bf16, ub):
    x, res, w = make(m, k, bf16, seed=m * 5 + k)
    t_ub = None if ub is None else torch.full((1,), ub, device="cuda")
    got = qk.add_rmsnorm_quant_per_token_fp8(x_dev(x), x_dev(w), x_dev(res), 1e-6, scale_ub=t_ub, want_norm=True)
    check(O, x, res, w, 1e-6, got, fp8=True, ub=ub)


@pytest.mark.parametrize("m", [12, 600])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
def test_norm_special_rows(O, m, bf16, fp8):
    """Zero rows, rows under the floor, subnormal and very large values, ties."""
    k = 1024
    x, _, w = make(m, k, False, seed=9, residual=False)
    x[0] = 0.0
    x[1] = 1e-30
    x[2] *= 1e-20
    x[3] *= 2.0 ** 50
    x[4] *= 2.0 ** -140          # subnormal
    x[5] = 0.0
    x[5, 7] = 2.0 ** 40          # one value alone: rstd makes it sqrt(k)
    x[6] = 1.0
    w[:] = 1.0
    x[7] = np.arange(k) % 255 - 127.0   # codes of the row itself, so ...
    x[8] = (np.arange(k) % 254 - 126.5)  # ... every second is a tie once 127 is the largest
    x[8, 0] = 127.0
    x, w = as_type(x, bf16), as_type(w, bf16)
    fn = qk.add_rmsnorm_quant_per_token_fp8 if fp8 else qk.add_rmsnorm_quant_per_token
    got = fn(x_dev(x), x_dev(w), eps=1e-6, want_norm=True)
    check(O, x, None, w, 1e-6, got, fp8=fp8)
    assert not host(got[0])[0].any() and host(got[1])[0] == np.float32(1e-12) / np.float32(448 if fp8 else 127)


@pytest.mark.parametrize("m,k", [(5, 528), (600, 4096), (2, 140000)])
@pytest.mark.parametrize("into", ["residual", "x", "other"])
def test_norm_in_place_and_strides(O, m, k, into):
    """residual_out over one of its inputs, and rows that lie in a wider buffer."""
    x, res, w = make(m, k, True, seed=m + k + 1)
    wide = torch.full((m, k + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + k] = x_dev(x)
    xs = wide[:, 8:8 + k]
    rs = x_dev(res)
    out = {"residual": rs, "x": xs, "other": None}[into]
    got = qk.add_rmsnorm_quant_per_token(xs, x_dev(w), rs, 1e-6, want_norm=True, residual_out=out)
    if out is not None:
        assert got[2].data_ptr() == out.data_ptr()
    check(O, x, res, w, 1e-6, got)
    if into != "x":
        assert torch.equal(xs, x_dev(x))
    assert bool((wide[:, :8] == 7.0).all()) and bool((wide[:, 8 + k:] == 7.0).all())


@pytest.mark.parametrize("m,k", [(6, 4096), (700, 1024)])
def test_norm_bad_row_stays_alone(m, k):
    x, res, w = make(m, k, True, seed=3)
    xd, rd, wd = x_dev(x), x_dev(res), x_dev(w)
    clean = qk.add_rmsnorm_quant_per_token(xd, wd, rd, want_norm=True)
    xd[2, 5] = float("nan")
    xd[4, 9] = float("inf")
    dirty = qk.add_rmsnorm_quant_per_token(xd, wd, rd, want_norm=True)
    keep = [i for i in range(m) if i not in (2, 4)]
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])


def test_norm_rows_do_not_depend_on_the_batch():
    """A row's result is the same alone and among many: the forms for few and many rows agree bit for bit
    in what depends on no sum, and repeated calls agree in everything."""
    x, res, w = make(800, 4096, True, seed=21)
    xd, rd, wd = x_dev(x), x_dev(res), x_dev(w)
    many = qk.add_rmsnorm_quant_per_token(xd, wd, rd)
    again = qk.add_rmsnorm_quant_per_token(xd, wd, rd)
    for a, b in zip(many[:3], again[:3]):
        assert torch.equal(a, b)
    one = qk.add_rmsnorm_quant_per_token(xd[17:18], wd, rd[17:18])
    assert torch.equal(one[0], many[0][17:18]) and torch.equal(one[2], many[2][17:18])


def test_norm_helper_refusals():
    need_gpu()
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    good = lambda **kw: qk.add_rmsnorm_quant_per_token(**{**dict(x=x, weight=w), **kw})  # noqa: E731
    good()
    for kw in (dict(weight=w.float()), dict(weight=w[:32]), dict(residual=x.float()), dict(residual=x[:2]),
               dict(x=x.t()), dict(x=x[0]), dict(residual_out=x), dict(residual=x, residual_out=x[:, :32]),
               dict(norm_out=x[:, ::2]), dict(q=x), dict(scale=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            good(**kw)
    with pytest.raises(qk.QKError):
        good(eps=0.0)
    with pytest.raises(qk.QKError):
        good(x=torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")[:, :64][:, 4:60], weight=w[:56])
    q, s, r, n = qk.add_rmsnorm_quant_per_token(x[:0], w, x[:0], want_norm=True)
    assert q.shape == (0, 64) and s.shape == (0,) and r.shape == (0, 64) and n.shape == (0, 64)
