"""moe_grouped_gemm and its two gradients on the GPU against 64-bit products of the same inputs.

Tolerance, element by element: a 16-bit result is rounded once (half a step, eps/2 of the value, or half
the smallest subnormal); the fp32 sum under it is a chain of at most n additions, each off by at most
2^-23 of the sum of |a||b| (the tensor core truncates), where n is the contracted length plus one
alignment per 16-long instruction.  Results that stay fp32 are drained every 512 terms and added with
rounding, so there n is at most 512 + 32, plus 2^-24 per drain."""
import json
import os
import subprocess
import sys

import pytest
import torch

import sparse_mixture_experts_16_b200 as moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -149}


def sum_bound(n, promoted):
    if not promoted:
        return (n + n / 16 + 1) * 2.0 ** -23
    return (min(n, 512) * (1 + 1 / 16) + 1) * 2.0 ** -23 + (n / 512 + 17) * 2.0 ** -24


def close(got, ref, mag, n):
    """got (any type) against ref (64 bits), mag = sum of |a||b|, n terms per sum"""
    t = got.dtype
    err = (got.double() - ref).abs()
    lim = sum_bound(n, t == F32) * mag
    if t != F32:
        lim = lim + torch.finfo(t).eps / 2 * (ref.abs() + lim) + TINY[t]
    bad = ~(err <= lim)
    assert not bad.any(), (int(bad.sum()), float(err.max()), float((err - lim).max()))


def offsets_of(counts, first=0):
    edges = [first]
    for c in counts:
        edges.append(edges[-1] + c)
    return torch.tensor(edges, dtype=torch.int32, device="cuda")


def data(seed, M, E, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    dy = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    w = (torch.randn(E, N, K, generator=g, device="cuda") * K ** -0.5).to(dtype)
    return x, dy, w


def check_all(counts, N, K, dtype, out_dtype, first=0, behind=0, seed=0):
    """The three operators on one routing; rows before the first and behind the last segment keep a mark."""
    E = len(counts)
    off = offsets_of(counts, first)
    M = first + sum(counts) + behind
    x, dy, w = data(seed, M, E, N, K, dtype)
    edges = off.tolist()
    y = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    dx = torch.full((M, K), 7.0, dtype=out_dtype, device="cuda")
    _, ws = moe.moe_grouped_gemm(x, off, w, out=y)
    moe.moe_grouped_gemm_dgrad(dy, off, w, out=dx, ws=ws)
    dw, ws2 = moe.moe_grouped_gemm_wgrad(dy, x, off)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0 and moe.moe_get_device_error(ws2) == 0
    xd, dyd, wd = x.double(), dy.double(), w.double()
    for e in range(E):
        s = slice(edges[e], edges[e + 1])
        close(y[s], xd[s] @ wd[e].T, xd[s].abs() @ wd[e].abs().T, K)
        close(dx[s], dyd[s] @ wd[e], dyd[s].abs() @ wd[e].abs(), N)
        close(dw[e], dyd[s].T @ xd[s], dyd[s].T.abs() @ xd[s].abs(), edges[e + 1] - edges[e])
    for t in (y, dx):
        assert (t[:first] == 7.0).all() and (t[M - behind:] == 7.0).all()


ROUTINGS = {
    "one_row": [1],
    "one_token_top4": [0, 1, 0, 0, 1, 1, 0, 1],
    "empty_between": [0, 130, 0, 0, 1, 64, 0],
    "all_to_one": [0, 0, 700, 0],
    "tile_edges": [255, 256, 257, 15, 16, 17, 1],
    "block_edges": [63, 64, 65, 127, 128, 129, 31],
}


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (HF, HF), (BF, F32), (HF, F32)],
                         ids=["bf16", "fp16", "bf16_f32", "fp16_f32"])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 200), (264, 520), (512, 256)])
@pytest.mark.parametrize("routing", list(ROUTINGS))
def test_products(cuda_device, routing, N, K, dtype, out_dtype):
    check_all(ROUTINGS[routing], N, K, dtype, out_dtype, seed=N + K)


@pytest.mark.parametrize("counts,N,K,dtype,out_dtype", [
    ([1, 0, 1, 1, 1], 2880, 1440, BF, BF),        # one token: split along K
    ([3, 1, 0, 2, 9] * 6, 1000, 2048, HF, F32),
    ([900, 30, 0, 2100], 1024, 776, BF, BF),      # several bands of row tiles
    ([2500], 264, 136, HF, HF),                   # more than 8 row tiles of one expert
    ([5] * 1024, 16, 24, BF, F32),                # the most experts
    ([5000, 3], 520, 264, BF, F32),               # long segments: many drains
], ids=["token", "ragged", "bands", "one_expert", "experts_1024", "long"])
def test_larger_products(cuda_device, counts, N, K, dtype, out_dtype):
    check_all(counts, N, K, dtype, out_dtype, seed=3)


def test_rows_outside_the_segments_keep_what_they_held(cuda_device):
    check_all([10, 0, 40], 72, 64, BF, BF, first=5, behind=300)


def test_no_rows(cuda_device):
    x, dy, w = data(0, 0, 3, 16, 24, BF)
    off = offsets_of([0, 0, 0])
    y, _ = moe.moe_grouped_gemm(x, off, w)
    dx, _ = moe.moe_grouped_gemm_dgrad(dy, off, w)
    dw, _ = moe.moe_grouped_gemm_wgrad(dy, x, off, out=torch.full((3, 16, 24), 5.0, device="cuda"))
    assert y.shape == (0, 16) and dx.shape == (0, 24) and (dw == 0).all()
    x, dy, w = data(0, 20, 3, 16, 24, BF)  # rows, but none of them in a segment
    y, _ = moe.moe_grouped_gemm(x, off, w, out=torch.full((20, 16), 5.0, device="cuda", dtype=BF))
    dw, _ = moe.moe_grouped_gemm_wgrad(dy, x, off, out=torch.full((3, 16, 24), 5.0, device="cuda"))
    assert (y == 5.0).all() and (dw == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_segments_do_not_see_infinities(cuda_device, bad):
    """segment 1 of three is full of NaN or infinities, and so is what lies outside the segments"""
    counts, N, K = [37, 50, 41], 136, 200
    off = offsets_of(counts, 3)
    edges = off.tolist()
    M = edges[-1] + 9
    x, dy, w = data(1, M, 3, N, K, BF)
    for t in (x, dy):
        t[:edges[0]] = bad
        t[edges[1]:edges[2]] = bad
        t[edges[3]:] = bad
    w[1] = bad
    y, _ = moe.moe_grouped_gemm(x, off, w)
    dx, _ = moe.moe_grouped_gemm_dgrad(dy, off, w)
    dw, _ = moe.moe_grouped_gemm_wgrad(dy, x, off)
    for e in (0, 2):
        s = slice(edges[e], edges[e + 1])
        close(y[s], x[s].double() @ w[e].double().T, x[s].double().abs() @ w[e].double().abs().T, K)
        close(dx[s], dy[s].double() @ w[e].double(), dy[s].double().abs() @ w[e].double().abs(), N)
        close(dw[e], dy[s].double().T @ x[s].double(), dy[s].double().T.abs() @ x[s].double().abs(), counts[e])
    assert not torch.isfinite(dw[1]).any()


@pytest.mark.parametrize("rows", [1024, 16384])
def test_long_fp32_sums_keep_fp32_accuracy(cuda_device, rows):
    """all terms positive: truncation would bias the sum by about 5e-9 per term (8e-5 at 16384).  With a
    drain every 512 terms: 32 truncations of at most 2^-23 of a piece that is half full on average, and
    rounded additions: below 2e-6 + 2^-24 * drains."""
    x, dy, _ = data(2, rows, 1, 128, 128, BF)
    x, dy = x.abs(), dy.abs()
    dw, _ = moe.moe_grouped_gemm_wgrad(dy, x, offsets_of([rows]))
    ref = dy.double().T @ x.double()
    assert float((dw[0].double() - ref).norm() / ref.norm()) < 2e-6 + rows / 512 * 2.0 ** -24
    y, _ = moe.moe_grouped_gemm(x.T.contiguous(), offsets_of([128]), dy.T.contiguous()[None], out_dtype=F32)
    ref = x.double().T @ dy.double()
    assert float((y.double() - ref).norm() / ref.norm()) < 2e-6 + rows / 512 * 2.0 ** -24


def test_gradients_against_differences(cuda_device):
    """L = sum(r * y): dgrad and wgrad against central differences of the forward in 64 bits.  L is
    bilinear, so the differences are exact but for 64-bit rounding."""
    counts, N, K = [5, 0, 9], 24, 40
    off = offsets_of(counts)
    edges = off.tolist()
    x, r, w = data(4, 14, 3, N, K, BF)
    dx, _ = moe.moe_grouped_gemm_dgrad(r, off, w, out_dtype=F32)
    dw, _ = moe.moe_grouped_gemm_wgrad(r, x, off)

    def loss(xd, wd):
        return sum((r[edges[e]:edges[e + 1]].double() * (xd[edges[e]:edges[e + 1]] @ wd[e].T)).sum() for e in range(3))

    g = torch.Generator().manual_seed(0)
    xd, wd, h = x.double(), w.double(), 0.5
    for _ in range(20):
        i, j = int(torch.randint(14, (1,), generator=g)), int(torch.randint(K, (1,), generator=g))
        e, n = int(torch.randint(3, (1,), generator=g)), int(torch.randint(N, (1,), generator=g))
        px, mx, pw, mw = xd.clone(), xd.clone(), wd.clone(), wd.clone()
        px[i, j] += h
        mx[i, j] -= h
        pw[e, n, j] += h
        mw[e, n, j] -= h
        for got, ref, size in ((dx[i, j], (loss(px, wd) - loss(mx, wd)) / (2 * h), N),
                               (dw[e, n, j], (loss(xd, pw) - loss(xd, mw)) / (2 * h), counts[e])):
            # terms below about 16 in size: (n + 2) truncations of 2^-23 of at most 16 n
            assert abs(float(got) - float(ref)) <= (size + 2) * 2.0 ** -23 * 16 * max(1, size) + 1e-9


def test_results_do_not_depend_on_timing(cuda_device):
    """few rows: parts of K are added by whichever part arrives last, always in the order of the parts"""
    counts = [1, 0, 2, 1, 0, 4]
    off = offsets_of(counts)
    x, dy, w = data(5, 8, 6, 1000, 1504, BF)
    first, ws = moe.moe_grouped_gemm(x, off, w, out_dtype=F32)
    for _ in range(20):
        again, _ = moe.moe_grouped_gemm(x, off, w, out_dtype=F32, ws=ws)
        assert torch.equal(first, again)


def test_streams_and_a_shared_workspace(cuda_device):
    """calls of different sizes in turn on one side stream and one workspace"""
    s = torch.cuda.Stream()
    ws = torch.zeros(moe.lib().moe_grouped_gemm_workspace_size(4096), dtype=torch.uint8, device="cuda")
    got = []
    sizes = [([1, 2, 0], 264, 1024), ([300, 5, 90], 72, 64), ([4, 4, 4], 1000, 520)]
    args = [(offsets_of(c), *data(i, sum(c), 3, N, K, HF)) for i, (c, N, K) in enumerate(sizes)]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for off, x, dy, w in args * 2:
            got.append((moe.moe_grouped_gemm(x, off, w, ws=ws)[0], moe.moe_grouped_gemm_dgrad(dy, off, w, ws=ws)[0],
                        moe.moe_grouped_gemm_wgrad(dy, x, off, ws=ws)[0]))
    s.synchronize()
    for i, (off, x, dy, w) in enumerate(args * 2):
        alone = (moe.moe_grouped_gemm(x, off, w)[0], moe.moe_grouped_gemm_dgrad(dy, off, w)[0],
                 moe.moe_grouped_gemm_wgrad(dy, x, off)[0])
        assert all(torch.equal(a, b) for a, b in zip(got[i], alone))


def test_captured_and_replayed_with_other_routing(cuda_device):
    """one captured graph serves every routing of the same number of rows: offsets are read on the device"""
    N, K, M, E = 136, 264, 60, 5
    x, dy, w = data(6, M, E, N, K, BF)
    off = offsets_of([12] * 5)
    y, ws = moe.moe_grouped_gemm(x, off, w)
    dw, ws2 = moe.moe_grouped_gemm_wgrad(dy, x, off)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_grouped_gemm(x, off, w, out=y, ws=ws)
        moe.moe_grouped_gemm_wgrad(dy, x, off, out=dw, ws=ws2)
    for counts in ([60, 0, 0, 0, 0], [1, 2, 3, 4, 50], [0, 0, 31, 0, 29]):
        off.copy_(offsets_of(counts))
        x.copy_(data(sum(counts[:2]), M, E, N, K, BF)[0])
        g.replay()
        edges = off.tolist()
        for e in range(E):
            s = slice(edges[e], edges[e + 1])
            close(y[s], x[s].double() @ w[e].double().T, x[s].double().abs() @ w[e].double().abs().T, K)
            close(dw[e], dy[s].double().T @ x[s].double(), dy[s].double().T.abs() @ x[s].double().abs(), counts[e])


@pytest.mark.parametrize("edges", [[0, 10, 5, 20], [-4, 3, 8, 20], [0, 3, 8, 400]])
def test_bad_offsets_are_reported_and_stay_in_bounds(cuda_device, edges):
    M, N, K = 20, 40, 24
    x, dy, w = data(7, M, 3, N, K, BF)
    off = torch.tensor(edges, dtype=torch.int32, device="cuda")
    room = torch.full((M + 64, N), 3.0, dtype=BF, device="cuda")
    _, ws = moe.moe_grouped_gemm(x, off, w, out=room[:M])
    assert moe.moe_get_device_error(ws) == 6  # MOE_ERR_DEVICE_INDEX
    assert moe.moe_get_device_error(ws) == 0  # read once
    assert (room[M:] == 3.0).all()
    _, ws = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert moe.moe_get_device_error(ws) == 6


def test_refusals(cuda_device):
    x, dy, w = data(8, 12, 2, 16, 24, BF)
    off = offsets_of([5, 7])
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x[:, ::2], off, w)                   # strided rows
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off.long(), w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off[:-1].contiguous(), w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off, w.half())
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_dgrad(x, off, w)                     # x is K wide, not N
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_wgrad(dy[:5], x, off)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off, w, out=torch.empty(12, 16, device="cuda", dtype=HF))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x.cpu(), off, w)
    with pytest.raises(moe.MoeError):
        moe.moe_grouped_gemm(x[:, :20].contiguous(), off, w[..., :20].contiguous())  # K not a multiple of 8


CHILD = r"""
import json, sys, time
sys.path.insert(0, {root!r})
import torch
import sparse_mixture_experts_16_b200 as moe
torch.manual_seed(0)
op = {op!r}
x = torch.randn(300, 256, device="cuda").bfloat16()
dy = torch.randn(300, 128, device="cuda").bfloat16()
w = torch.randn(2, 128, 256, device="cuda").bfloat16()
off = torch.tensor([0, 170, 300], dtype=torch.int32, device="cuda")
g = torch.randn(2, 200, 300, device="cuda")
def call(ws):
    if op == "gemm":
        return moe.moe_grouped_gemm(x, off, w, ws=ws)
    if op == "dgrad":
        return moe.moe_grouped_gemm_dgrad(dy, off, w, ws=ws)
    if op == "wgrad":
        return moe.moe_grouped_gemm_wgrad(dy, x, off, ws=ws)
    return moe.moe_orthogonalize(g, ws=ws)
torch.cuda.synchronize()
t0 = time.time()
out, ws = call(None)               # its first launch withholds its first copies
torch.cuda.synchronize()
elapsed = time.time() - t0
first = moe.moe_get_device_error(ws)
ws.zero_()
out, ws = call(ws)
second = moe.moe_get_device_error(ws)
ref, _ = call(None)
print("RESULT " + json.dumps(dict(first=first, second=second, elapsed=elapsed, same=bool(torch.equal(out, ref)))))
"""


@pytest.mark.parametrize("op", ["gemm", "dgrad", "wgrad", "ortho"])
def test_withheld_copy_times_out_and_the_context_stays_usable(cuda_device, op):
    env = dict(os.environ, MOE_TEST_WITHHOLD_LOAD="1")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, op=op)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads([ln for ln in r.stdout.splitlines() if ln.startswith("RESULT ")][-1][len("RESULT "):])
    assert res["first"] == 7 and res["second"] == 0 and res["same"] and res["elapsed"] < 60


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [
    ([511, 513, 1040, 300, 0, 769], 264, 200),   # rows dealt evenly over the tiles
    ([2049], 520, 72),
    ([42], 9264, 96), ([42], 96, 9264),          # one tile, split along a long axis
    ([0, 3, 0, 0, 28, 0, 0, 1], 136, 8136),
    ([3, 5, 2], 24, 4000),
    ([1300], 24, 2008),                          # a long segment, a narrow gradient
    ([190] * 8, 1000, 520),
], ids=["even", "one", "long_n", "long_k", "ragged_long_k", "few", "narrow", "half_a_round"])
def test_tiles_and_parts(cuda_device, counts, N, K, out_dtype):
    check_all(counts, N, K, BF, out_dtype, seed=11)


def test_outputs_past_32_bits(cuda_device):
    """2^31 elements and more: the last rows, the last expert"""
    M, N, K, E = 70016, 32768, 16, 2
    x, dy, w = data(9, M, 1, 8, K, BF)[0], None, data(10, 8, E, N, K, BF)[2]
    off = offsets_of([69000, 1016])
    y, ws = moe.moe_grouped_gemm(x, off, w)
    assert y.numel() > 2 ** 31 and moe.moe_get_device_error(ws) == 0
    for e, s in ((0, slice(0, 40)), (0, slice(68960, 69000)), (1, slice(69000, 69040)), (1, slice(69976, 70016))):
        a, b = x[s].double(), w[e].double()
        close(y[s], a @ b.T, a.abs() @ b.abs().T, K)
    del y
    E, N, K = 33, 8192, 8192
    dy, x = data(12, 66, 1, N, K, BF)[1], data(13, 66, 1, N, K, BF)[0]
    off = offsets_of([2] * E)
    dw, ws = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert dw.numel() > 2 ** 31 and moe.moe_get_device_error(ws) == 0
    for e in (0, 31, 32):
        a, b = dy[2 * e:2 * e + 2].double().T, x[2 * e:2 * e + 2].double()
        close(dw[e], a @ b, a.abs() @ b.abs(), 2)


def test_a_segment_that_takes_longer_than_a_wait(cuda_device):
    """2^29 + 3 rows in one of 100 segments, whose tile is not split: the wait for its last block would expire.
    The products are -1, 0 or 1 and their sums stay far below 2^24, so that every order of adding is exact."""
    E, M, N, K = 100, 2 ** 29 + 3, 8, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.empty(M, K, dtype=BF, device="cuda").random_(-1, 2, generator=g)
    dy = torch.empty(M, N, dtype=BF, device="cuda").random_(-1, 2, generator=g)
    off = offsets_of([M] + [0] * (E - 1))
    dw, ws = moe.moe_grouped_gemm_wgrad(dy, x, off)
    assert moe.moe_get_device_error(ws) == 0
    ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for at in range(0, M, 2 ** 24):
        ref += dy[at:at + 2 ** 24].double().T @ x[at:at + 2 ** 24].double()
    assert ref.abs().max() < 2 ** 24
    assert torch.equal(dw[0].double(), ref) and not dw[1:].any()


def test_two_streams_with_a_workspace_each(cuda_device):
    """calls that run side by side, each on its own stream and workspace, give what they give alone"""
    off = offsets_of([100, 3, 0, 500])
    x, dy, w = data(14, 603, 4, 520, 776, BF)
    alone = [moe.moe_grouped_gemm(x, off, w)[0], moe.moe_grouped_gemm_dgrad(dy, off, w)[0],
             moe.moe_grouped_gemm_wgrad(dy, x, off)[0]]
    streams = [torch.cuda.Stream() for _ in range(3)]
    wss = [None, None, None]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for i, st in enumerate(streams):
            call = [lambda **k: moe.moe_grouped_gemm(x, off, w, **k), lambda **k: moe.moe_grouped_gemm_dgrad(dy, off, w, **k),
                    lambda **k: moe.moe_grouped_gemm_wgrad(dy, x, off, **k)][i]
            if wss[i] is None:
                with torch.cuda.stream(st):
                    out, wss[i] = call()
            else:
                with torch.cuda.stream(st):
                    out, _ = call(ws=wss[i], stream=st)
            got.append(out)
        for st in streams:
            st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone))


def test_the_same_rows_in_two_operands(cuda_device):
    """x and dy may be one tensor, and an output may be reused by the next call"""
    off = offsets_of([70, 0, 60])
    x = data(15, 130, 3, 136, 136, BF)[0]
    dw, ws = moe.moe_grouped_gemm_wgrad(x, x, off)
    for e, s in ((0, slice(0, 70)), (2, slice(70, 130))):
        a = x[s].double()
        close(dw[e], a.T @ a, a.abs().T @ a.abs(), s.stop - s.start)
    kept = dw.clone()
    out, _ = moe.moe_grouped_gemm_wgrad(x, x, off, out=dw, ws=ws)
    assert out is dw and torch.equal(dw, kept)


def test_unaligned_and_small_workspaces_are_refused(cuda_device):
    x, dy, w = data(16, 12, 2, 16, 24, BF)
    off = offsets_of([5, 7])
    shifted = torch.empty(12 * 24 + 1, dtype=BF, device="cuda")[1:].view(12, 24)
    with pytest.raises(moe.MoeError, match="ALIGNMENT"):
        moe.moe_grouped_gemm(shifted, off, w)
    small = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    _, ws = moe.moe_grouped_gemm(x, off, w, ws=small)  # too small: another one comes back
    assert ws is not small
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, off, w, ws=torch.zeros(1 << 26, dtype=torch.float32, device="cuda"))


def test_what_a_call_allocates_belongs_to_its_stream(cuda_device):
    """the workspace's zeroing and the output of a call with ``stream`` are ordered on that stream, whatever
    the current one is busy with"""
    off = offsets_of([4, 0, 9])
    x, dy, w = data(17, 13, 3, 1000, 1504, BF)
    want = moe.moe_grouped_gemm(x, off, w, out_dtype=F32)[0], moe.moe_orthogonalize(w.float())[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda._sleep(20_000_000)  # the current stream is behind
        y, ws = moe.moe_grouped_gemm(x, off, w, out_dtype=F32, stream=side)
        side.synchronize()
        assert torch.equal(y, want[0]) and moe.moe_get_device_error(ws, side) == 0
    wf = w.float()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    u, _ = moe.moe_orthogonalize(wf, stream=side)
    side.synchronize()
    assert torch.equal(u, want[1])
