"""moe_add_rms_norm on the GPU against 64 bits (needs an MI355X).

Tolerances.  s = x + residual is one fp32 addition (2^-24 relative), residual_out one more rounding.  y: the sum
of squares adds at most H/256 + 64 terms one after another (a thread's own, its wave's and workgroup's trees),
every term off by 3 * 2^-24 relative at most, so sqrt halves (H/256 + 67) * 2^-24; the division, square root and
two products add 5 * 2^-24.  That is below REL(H) = (H/256 + 80) * 2^-24, plus half a step of y's type (and half
the smallest subnormal, 2^-25, for fp16)."""
import numpy as np
import pytest
import torch

import front_reference as ref
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rel(H):
    return (H / 256 + 80) * 2.0 ** -24


def near(got, want, r, tiny):
    got = got.float().cpu().numpy().astype(np.float64)
    bad = np.abs(got - want) > np.abs(want) * r + tiny
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def check(T, H, x, res, y, w, mx, seed=0, scale=1.0, eps=1e-6, pad=0, in_place=False):
    note(f"norm T={T} H={H} x={x} residual={res} y={y} weight={w} mx={mx} pad={pad}")
    g = torch.Generator().manual_seed(seed)
    rows = lambda t: torch.randn(T, H + pad, generator=g).mul(scale).to(TYPES[t]).to(DEV)[:, :H]
    X, R = rows(x), None if res is None else rows(res)
    Wt = (1 + 0.2 * torch.randn(H, generator=g)).to(TYPES[w]).to(DEV)
    s, want = ref.add_rms_norm(X.double().cpu().numpy(), None if R is None else R.double().cpu().numpy(),
                               Wt.double().cpu().numpy(), eps)
    norm = moe.RmsNorm(Wt, eps)
    if in_place:
        Y = torch.empty(T, H, dtype=TYPES[y], device=DEV)
        codes = torch.empty(T, moe.moe_mx_row_bytes(mx, H), dtype=torch.uint8, device=DEV) if mx else None
        scales = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV) if mx else None
        out = moe.moe_add_rms_norm(X, norm, R, mx=mx, out=(Y, R, codes, scales))
        assert out[1] is R
    else:
        out = moe.moe_add_rms_norm(X, norm, R, mx=mx, dtype=TYPES[y])
    torch.cuda.synchronize()
    Y, RO, codes, scales = out
    assert Y.dtype == TYPES[y]
    tiny = lambda t: 2.0 ** -25 if t == "fp16" else 0.0
    near(Y, want, rel(H) + ref.half_step(y) * (1 + rel(H)), tiny(y))
    if res is None:
        assert RO is None
    else:
        assert RO.dtype == TYPES[res]
        near(RO, s, 2.0 ** -24 + ref.half_step(res) * (1 + 2.0 ** -24), tiny(res))
    if mx:
        ref.check_mx(want, codes.cpu().numpy(), scales.cpu().numpy(), mx, rel(H))


SIZES = [(1, 32), (3, 64), (2, 480), (5, 512), (7, 2048), (4, 2080), (2, 4096), (3, 7168), (2, 8192), (2, 8224),
         (2, 16384), (1, 16416), (1, 32768), (1, 32800), (130, 96)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("mx", [None, "fp8", "fp6", "fp4"])
def test_lengths(T, H, mx):
    check(T, H, "fp32", "bf16", "bf16", "bf16", mx, seed=H)


@pytest.mark.parametrize("T,H", [(1, 1), (2, 7), (3, 33), (5, 255), (2, 257), (3, 4097), (1, 33001), (64, 40)])
def test_odd_lengths(T, H):
    check(T, H, "fp16", "fp16", "fp16", "fp32", None, seed=H)


@pytest.mark.parametrize("x", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("res", [None, "bf16", "fp16", "fp32"])
@pytest.mark.parametrize("y,w,H", [("bf16", "fp32", 1024), ("fp16", "bf16", 1024), ("fp32", "fp16", 1024),
                                   ("fp32", "bf16", 91)])
def test_types(x, res, y, w, H):
    check(3, H, x, res, y, w, "fp8" if H % 32 == 0 else None, seed=3)


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("H", [256, 2048])
@pytest.mark.parametrize("mx", [None, "fp8", "fp6"])
def test_in_place_and_strided(H, pad, mx):
    check(5, H, "bf16", "bf16", "bf16", "bf16", mx, seed=pad, pad=pad, in_place=True)


@pytest.mark.parametrize("H", [5, 9, 63, 257, 513, 4097, 8191, 16411, 32769])
@pytest.mark.parametrize("pad", [0, 2])
def test_in_place_odd(H, pad):
    """The last run of a row overlaps the one before: in place, no value may be added twice."""
    check(3, H, "fp16", "fp16", "fp16", "bf16", None, seed=H, pad=pad, in_place=True)
    check(2, H, "bf16", "fp32", "fp32", "fp32", None, seed=H, pad=pad, in_place=True)


@pytest.mark.parametrize("H", [512, 513])
def test_scales_of_values(H):
    check(4, H, "fp32", "fp32", "fp32", "fp32", None, scale=1e-12, eps=1e-30)
    check(4, H, "fp32", "fp32", "fp32", "fp32", None, scale=1e15)
    check(4, H, "bf16", "bf16", "bf16", "bf16", None, scale=1e-3, eps=1e-2)  # eps outweighs the mean square


def test_zero_rows():
    """A row of zeros: y is 0 (not NaN) for a positive eps, codes are 0 with scale code 0."""
    X = torch.zeros(3, 64, device=DEV)
    X[1] = 1.0
    Y, RO, codes, scales = moe.moe_add_rms_norm(X, moe.RmsNorm(torch.ones(64, device=DEV)), torch.zeros_like(X), mx="fp8")
    assert torch.equal(Y[0].float(), torch.zeros(64, device=DEV)) and int(codes[0].sum()) == 0
    assert int(scales[0].sum()) == 0 and torch.equal(RO, X)
    near(Y[1:2], np.full((1, 64), 1 / np.sqrt(1 + 1e-6)), 2.0 ** -8 + rel(64), 0.0)


def test_nothing_else_is_written():
    """Rows and columns outside the outputs keep their contents."""
    T, H = 5, 96
    for pad in (8, 5):
        buf = torch.full((T + 2, H + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        X = torch.randn(T, H, device=DEV)
        R = torch.randn(T, H, device=DEV).bfloat16()
        Y = torch.full((T + 2, H), 7.0, dtype=torch.float32, device=DEV)
        moe.moe_add_rms_norm(X, moe.RmsNorm(torch.ones(H, device=DEV)), R, out=(Y[1:1 + T], buf[1:1 + T, :H], None, None))
        assert bool((buf[0] == 7).all() & (buf[-1] == 7).all() & (buf[:, H:] == 7).all())
        assert bool((Y[0] == 7).all() & (Y[-1] == 7).all())
        assert torch.equal(buf[1:1 + T, :H], (X + R.float()).bfloat16())


def test_outputs_left_out():
    X = torch.randn(4, 256, device=DEV)
    norm = moe.RmsNorm(torch.ones(256, device=DEV))
    full = moe.moe_add_rms_norm(X, norm, X, mx="fp8")
    codes, scales = torch.zeros_like(full[2]), torch.zeros_like(full[3])
    y, ro, _, _ = moe.moe_add_rms_norm(X, norm, X, mx="fp8", out=(None, None, codes, scales))
    assert y is None and ro is None and torch.equal(codes, full[2]) and torch.equal(scales, full[3])


def test_empty_batch():
    X = torch.empty(0, 256, device=DEV)
    y, ro, codes, scales = moe.moe_add_rms_norm(X, moe.RmsNorm(torch.ones(256, device=DEV)), X, mx="fp8")
    assert y.shape == (0, 256) and codes.shape == (0, 256)


def test_other_stream_and_repeat():
    """A call on a side stream, and the same bits on every run."""
    X = torch.randn(200, 4096, device=DEV)
    R = torch.randn(200, 4096, device=DEV).bfloat16()
    norm = moe.RmsNorm(torch.rand(4096, device=DEV))
    a = moe.moe_add_rms_norm(X, norm, R, mx="fp8")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = moe.moe_add_rms_norm(X, norm, R, mx="fp8")
    torch.cuda.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("H", [256, 263, 4096, 5])
def test_rows_that_are_not_finite_stay_alone(H):
    """A NaN makes its row NaN; an infinity gives NaN where it stands and 0 beside it (its mean square is infinite);
    the other rows do not change."""
    T = 6
    X = torch.randn(T, H, device=DEV)
    R = torch.randn(T, H, device=DEV).bfloat16()
    norm = moe.RmsNorm(torch.rand(H, device=DEV) + 0.5)
    a = moe.moe_add_rms_norm(X, norm, R)
    X2 = X.clone()
    X2[1, H - 1], X2[4, 2] = float("nan"), float("inf")
    b = moe.moe_add_rms_norm(X2, norm, R)
    keep = [0, 2, 3, 5]
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])
    assert bool(torch.isnan(b[0][1]).all()) and torch.isnan(b[0][4]).nonzero().flatten().tolist() == [2]
    assert int(torch.count_nonzero(b[0][4])) == 1 and bool(torch.isinf(b[1][4, 2])) and bool(torch.isnan(b[1][1, H - 1]))
