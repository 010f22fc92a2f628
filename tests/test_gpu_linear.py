"""moe_linear on the GPU against 64 bits (needs an MI355X); the tolerance is derived at
front_reference.linear_tolerance."""
import numpy as np
import pytest
import torch

import front_reference as ref
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = ["mxfp4", "int4g32", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def check(T, N, K, fmt, y="fp32", bias=False, xpad=0, ypad=0, seed=0, std=1.0):
    note(f"linear T={T} N={N} K={K} {fmt} -> {y} bias={bias} pads {xpad} {ypad}")
    rng = np.random.default_rng(seed + 7 * N + K)
    codes, scales, zeros, ts, w = ref.weights(fmt, N, K, rng)
    X = torch.from_numpy(rng.standard_normal((T, K + xpad)) * std).bfloat16()[:, :K]
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    x = X.double().numpy()
    want = x @ w.T + (0.0 if b is None else b.astype(np.float64))
    W = moe.LinearWeights(dev(codes), dev(scales), fmt, dev(zeros), dev(ts))
    xd = torch.empty_strided(X.shape, X.stride(), dtype=X.dtype, device=DEV).copy_(X)
    buf = torch.full((T + 2, N + ypad), 77.0, dtype=TYPES[y], device=DEV)
    got = moe.moe_linear(xd, W, dev(b), out=buf[1:-1, :N])
    torch.cuda.synchronize()
    assert bool((buf[0] == 77).all() & (buf[-1] == 77).all() & (buf[:, N:] == 77).all())
    got = got.double().cpu().numpy()
    tol = ref.linear_tolerance(x, w, K, want, y)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [32, 64, 96, 160, 480, 512, 544, 1056, 2080, 4096])
def test_inner_lengths(fmt, K):
    for T, N in ((1, 40), (5, 33), (40, 17), (130, 40)):
        check(T, N, K, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N", [1, 2, 15, 16, 31, 100, 257, 1000])
def test_outer_lengths(fmt, N):
    for T in (1, 16, 200):
        check(T, N, 160, fmt, "bf16", bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 32, 33, 47, 48, 49, 64, 65, 96, 127, 128, 129, 256, 300, 513])
def test_tokens(fmt, T):
    check(T, 72, 288, fmt)
    check(T, 130, 1024, fmt, "bf16")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("y", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("xpad,ypad", [(0, 0), (8, 1), (24, 16)])
def test_types_and_strides(fmt, y, xpad, ypad):
    for T in (1, 20, 140):
        check(T, 90, 192, fmt, y, bias=ypad > 0, xpad=xpad, ypad=ypad, std=2.0 ** -8)


@pytest.mark.parametrize("fmt", FORMATS)
def test_large(fmt):
    check(1, 4096, 7168, fmt)
    check(9, 1024, 7168, fmt, "bf16")
    check(192, 1280, 2048, fmt, "bf16", bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 20, 150])
def test_slices(fmt, T):
    """Rows and columns of a larger matrix (whole blocks, 16-byte steps), with scale rows at odd addresses."""
    rng = np.random.default_rng(5)
    N, K = 80, 640
    codes, scales, zeros, ts, w = ref.weights(fmt, N, K, rng)
    per = {"mxfp4": 1, "int4g32": 2, "nvfp4": 2}[fmt]  # scale bytes per 32 values
    for n0, n1, k0, k1 in ((3, 40, 96 * 2, 640), (16, 80, 64, 64 + 416), (0, 80, 64, 128)):
        b0, b1 = k0 // 32, k1 // 32
        W = moe.LinearWeights(dev(codes)[n0:n1, k0 // 2:k1 // 2], dev(scales)[n0:n1, b0 * per:b1 * per], fmt,
                              None if zeros is None else dev(zeros)[n0:n1, b0 // 2:(b1 + 1) // 2], dev(ts))
        X = torch.from_numpy(rng.standard_normal((T, k1 - k0))).bfloat16()
        x, ww = X.double().numpy(), w[n0:n1, k0:k1]
        want = x @ ww.T
        got = moe.moe_linear(X.to(DEV), W).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= ref.linear_tolerance(x, ww, k1 - k0, want, "fp32"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N", [(1, 2100), (3, 2049), (7, 6437), (9, 12850), (20, 6437), (25, 12850), (40, 6437),
                                 (50, 12850), (90, 6437), (700, 1030)])
def test_many_rows(fmt, T, N):
    check(T, N, 288, fmt, "bf16", bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(4, 3200, 96), (4, 3201, 96), (33, 70, 5120), (33, 70, 5152), (64, 130, 8192),
                                   (64, 6400, 5152), (50, 6420, 8192), (40, 6403, 8224), (32, 40, 9216),
                                   (16, 4096, 96), (10, 4097, 96), (16, 8192, 64), (5, 8193, 64), (32, 4096, 96),
                                   (17, 4097, 96), (20, 8193, 64), (31, 16385, 64), (33, 2048, 288), (65, 1366, 288),
                                   (129, 777, 544), (257, 910, 320), (513, 500, 288), (1025, 1000, 96),
                                   (1024, 1024, 4096), (1000, 1010, 4128), (40, 100, 12288), (35, 100, 12320),
                                   (2100, 33, 64), (300, 20, 12000)])
def test_where_kernels_meet(fmt, T, N, K):
    check(T, N, K, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3, 12, 30, 60, 150])
def test_scales_at_any_address(fmt, T):
    """Scale and zero-point rows at odd addresses, an odd number of bytes apart."""
    rng = np.random.default_rng(8)
    N, K = 50, 544
    codes, scales, zeros, ts, w = ref.weights(fmt, N, K, rng)

    def odd(a):
        if a is None:
            return None
        width = a.shape[1] + (2 if a.shape[1] % 2 else 1)
        buf = torch.zeros(1 + N * width, dtype=torch.uint8, device=DEV)
        view = buf[1:].view(N, width)[:, :a.shape[1]]
        view.copy_(dev(a))
        return view

    S, Z = odd(scales), odd(zeros)
    assert S.data_ptr() % 2 == 1 and S.stride(0) % 2 == 1
    X = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    x = X.double().numpy()
    want = x @ w.T
    got = moe.moe_linear(X.to(DEV), moe.LinearWeights(dev(codes), S, fmt, Z, dev(ts))).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= ref.linear_tolerance(x, w, K, want, "fp32"))


@pytest.mark.parametrize("T", [1, 20, 150])
def test_extreme_scales(T):
    """MXFP4 scale codes from the smallest to those whose sums fill fp32."""
    rng = np.random.default_rng(2)
    N, K = 32, 128
    codes, _, _, _, _ = ref.weights("mxfp4", N, K, rng)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(N, K)
    for e in (30, 100, 200, 240):
        scales = np.full((N, K // 32), e, np.uint8)
        w = ref.E2M1[c] * 2.0 ** (e - 127.0)
        X = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
        x = X.double().numpy()
        want = x @ w.T
        got = moe.moe_linear(X.to(DEV), moe.LinearWeights(dev(codes), dev(scales))).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= ref.linear_tolerance(x, w, K, want, "fp32"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3, 18, 130])
def test_a_row_that_is_not_finite_stays_alone(fmt, T):
    """NaN and infinities in one token's x reach that token's outputs only."""
    rng = np.random.default_rng(3)
    codes, scales, zeros, ts, _ = ref.weights(fmt, 50, 544, rng)
    W = moe.LinearWeights(dev(codes), dev(scales), fmt, dev(zeros), dev(ts))
    X = torch.from_numpy(rng.standard_normal((T, 544))).bfloat16().to(DEV)
    a = moe.moe_linear(X, W)
    X2 = X.clone()
    X2[T // 2, 17] = float("nan")
    X2[T // 2, 530] = float("inf")
    b = moe.moe_linear(X2, W)
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[T // 2]).all())


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_other_stream_and_repeat(T):
    rng = np.random.default_rng(11)
    codes, scales, _, _, _ = ref.weights("mxfp4", 512, 2048, rng)
    W = moe.LinearWeights(dev(codes), dev(scales))
    X = torch.from_numpy(rng.standard_normal((T, 2048))).bfloat16().to(DEV)
    a = moe.moe_linear(X, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = moe.moe_linear(X, W)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_empty_batch():
    rng = np.random.default_rng(1)
    codes, scales, _, _, _ = ref.weights("mxfp4", 8, 64, rng)
    assert moe.moe_linear(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV),
                          moe.LinearWeights(dev(codes), dev(scales))).shape == (0, 8)


def int4_weights(codes, zeros, scales):
    """LinearWeights of codes [N][K] and zero points [N][K/32] (four bits each) and binary16 scales [N][K/32]; and
    the decoded matrix in 64 bits."""
    N, K = codes.shape
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    z = np.pad(zeros, ((0, 0), (0, zeros.shape[1] % 2)))
    zp = (z[:, 0::2] | z[:, 1::2] << 4).astype(np.uint8)
    h = scales.astype(np.float16)
    w = (codes.astype(np.float64) - np.repeat(zeros, 32, 1)) * np.repeat(h.astype(np.float64), 32, 1)
    return moe.LinearWeights(dev(packed), dev(h.view(np.uint8).reshape(N, K // 16)), "int4g32", dev(zp)), w


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 20, 150])
@pytest.mark.parametrize("N,K", [(40, 4096), (2100, 288), (3210, 96)])
def test_int4_codes_at_their_zero_point(T, N, K):
    """Weights that are exactly zero add exactly nothing: rows of nothing else give 0 (or the bias), and the largest
    channels of x add no rounding where their code is the zero point."""
    rng = np.random.default_rng(T + N)
    zeros = rng.integers(0, 16, (N, K // 32))
    codes = np.repeat(zeros, 32, 1)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    b = rng.standard_normal(N).astype(np.float32)
    W, _ = int4_weights(codes, zeros, rng.uniform(0.005, 0.02, zeros.shape))
    assert not bool(moe.moe_linear(x.to(DEV), W).any())
    assert torch.equal(moe.moe_linear(x.to(DEV), W, dev(b)).cpu(), torch.from_numpy(b).expand(T, N))
    # one channel of each block 3000 times the others, its code the zero point; some of the other weights +-1 step
    step = rng.integers(-1, 2, (N, K)) * (rng.random((N, K)) < 0.2)
    big = np.arange(0, K, 32) + rng.integers(0, 32, K // 32)
    step[:, big] = 0
    codes = np.clip(codes + step, 0, 15)
    x[:, big] *= 3000
    W, w = int4_weights(codes, zeros, rng.uniform(0.005, 0.02, zeros.shape))
    xs = x.double().numpy()
    want = xs @ w.T
    got = moe.moe_linear(x.to(DEV), W).double().cpu().numpy()
    bad = ~(np.abs(got - want) <= ref.linear_tolerance(xs, w, K, want, "fp32"))
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("e", [0, 1, 2, 8, 29])
@pytest.mark.parametrize("T,N,K", [(1, 32, 128), (4, 40, 288), (20, 33, 128), (150, 32, 128), (1025, 1000, 96)])
def test_smallest_scale_codes(T, N, K, e):
    """MXFP4 scale codes from 2^-127 on, whose weights are bf16 subnormals, with x large enough for normal sums."""
    rng = np.random.default_rng(e)
    codes, _, _, _, _ = ref.weights("mxfp4", N, K, rng)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(N, K)
    scales = np.full((N, K // 32), e, np.uint8)
    w = ref.E2M1[c] * 2.0 ** (e - 127.0)
    X = torch.from_numpy(rng.standard_normal((T, K)) * 2.0 ** 100).bfloat16()
    x = X.double().numpy()
    want = x @ w.T
    got = moe.moe_linear(X.to(DEV), moe.LinearWeights(dev(codes), dev(scales))).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= ref.linear_tolerance(x, w, K, want, "fp32"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,K", [(16, 4097, 288), (5, 12288, 96), (9, 12289, 96), (16, 8192, 1312), (12, 8193, 1280),
                                   (7, 8193, 1312), (16, 16384, 1312), (6, 16385, 1312), (13, 24640, 1312)])
def test_rows_of_a_workgroup(fmt, T, N, K):
    """Up to 16 tokens on both sides of every change of the workgroups' rows."""
    check(T, N, K, fmt, "bf16")
