"""GPU checks of scored routing and of the float8 block-scaled operators against plain 64-bit forms
(scaled_ref), at the sizes and masks where they can go wrong, and of a run of them together."""
import numpy as np
import pytest

import scaled_ref as ref

from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

EPS = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}   # half a step


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    from expert_ffn_token_b200 import moe  # noqa: F401  (fails loudly if the library is missing)
    return t


@pytest.fixture(scope="module")
def moe(torch):
    from expert_ffn_token_b200 import moe as m
    return m


def _stream(torch):
    return torch.cuda.current_stream().cuda_stream


def _dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ scored routing

RULES = {
    "softmax": dict(score="softmax", renorm=True),
    "softmax kept": dict(score="softmax", renorm=False, scale=1.5),
    "softmax bias": dict(score="softmax", renorm=True, bias=0.01),
    "sigmoid": dict(score="sigmoid", renorm=False),
    "sigmoid bias": dict(score="sigmoid", renorm=True, scale=2.5, bias=0.3),
    "groups top1": dict(score="softmax", renorm=True, n_group=4, topk_group=2, group_top=1),
    "groups top1 bias": dict(score="sigmoid", renorm=True, n_group=4, topk_group=3, group_top=1,
                             bias=0.2),
    "groups top2": dict(score="sigmoid", renorm=True, n_group=4, topk_group=1, group_top=2),
    "groups top2 bias": dict(score="sigmoid", renorm=True, scale=2.5, n_group=4, topk_group=2,
                             group_top=2, bias=0.3),
}


def run_route(torch, moe, l, k, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True,
              scale=1.0, bias=None):
    T, E = l.shape
    ld = _dev(torch, l)
    bd = None if bias is None else _dev(torch, bias)
    new = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, counts, offs, perm, inv = new(T * k), new(E), new(E + 1), new(T * k), new(T * k)
    w = torch.full((T, k), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = moe.route_workspace_size(T, E, k)
    ws = torch.full((n,), 171, dtype=torch.uint8, device="cuda")
    rule = moe.RouteRule(moe.SCORE_SIGMOID if score == "sigmoid" else moe.SCORE_SOFTMAX, n_group,
                         topk_group, group_top, renorm, scale,
                         None if bd is None else bd.data_ptr())
    moe.route_scored(ld.data_ptr(), T, E, k, rule, ids.data_ptr(), w.data_ptr(), counts.data_ptr(),
                     offs.data_ptr(), perm.data_ptr(), inv.data_ptr(), status.data_ptr(),
                     ws.data_ptr(), n, _stream(torch))
    torch.cuda.synchronize()
    out = [t.cpu().numpy() for t in (ids.view(T, k), w, counts, offs, perm, inv)]
    return (*out, int(status.item()))


def check_route(torch, moe, l, k, rule):
    T, E = l.shape
    rule = dict(rule)
    ids, w, counts, offs, perm, inv, status = run_route(torch, moe, l, k, **rule)
    full = dict(score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0,
                bias=None)
    full.update(rule)
    rid, rw = ref.route(l, k, **full)
    assert status == 0
    assert np.array_equal(ids, rid)
    # the scores are 64-bit; a weight rounds to fp32 once (the normal range's half step, and
    # half the smallest subnormal below it); a softmax that is neither renormalised nor biased
    # divides by an fp32 sum: E / 32 additions in a row and exponentials 2 ulp off
    eps = 2.0 ** -23
    if full["score"] == "softmax" and not full["renorm"] and full["bias"] is None:
        eps += (E / 32 + 4) * 2.0 ** -24
    assert (np.abs(w - rw) <= eps * np.abs(rw) + 2.0 ** -149).all()
    rc, ro, rp, ri = ref.group(rid, E)
    assert np.array_equal(counts, rc) and np.array_equal(offs, ro)
    assert np.array_equal(perm, rp) and np.array_equal(inv, ri)


@pytest.mark.parametrize("name", list(RULES))
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (3, 512, 10), (17, 20, 3), (65, 64, 6),
                                   (300, 132, 12), (2, 4096, 32), (1500, 512, 10), (70, 1000, 16),
                                   (64, 1032, 8), (4100, 40, 4)])
def test_route_scored(torch, moe, name, T, E, k):
    rng = np.random.default_rng(T * 7919 + E + k)
    rule = dict(RULES[name])
    if "bias" in rule:
        rule["bias"] = (rule["bias"] * rng.standard_normal(E)).astype(np.float32)
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    check_route(torch, moe, l, k, rule)


@pytest.mark.parametrize("name", list(RULES))
def test_route_scored_ties_and_masks(torch, moe, name):
    """Logits on a coarse grid (ties go to the lower id), experts masked by the lowest fp32 value,
    rows with fewer open experts than k, rows with none, rows of one value."""
    T, E, k = 64, 64, 8
    rng = np.random.default_rng(5)
    l = np.round(2 * rng.standard_normal((T, E))).astype(np.float32)
    low = np.finfo(np.float32).min
    l[:16, rng.permutation(E)[:40]] = low
    l[16:24, 5:] = low
    l[24:28] = low
    l[28:32] = 3.0
    l[32:36] = 0.0
    l[36:40] = -90.0
    l[40:44] *= 20
    rule = dict(RULES[name])
    if "bias" in rule:
        rule["bias"] = (np.round(4 * rng.standard_normal(E)) / 8).astype(np.float32)
    check_route(torch, moe, l, k, rule)


@pytest.mark.parametrize("E", [64, 120, 2048])
@pytest.mark.parametrize("sign", [-1, 1])
def test_route_scored_group_sums_past_fp32(torch, moe, E, sign):
    """Biases near the type's limits: sums of two that pass fp32 are ranked as 64-bit ones."""
    rng = np.random.default_rng(E)
    bias = (sign * rng.uniform(1.8e38, 3.4e38, E)).astype(np.float32)
    l = (2 * rng.standard_normal((20, E))).astype(np.float32)
    check_route(torch, moe, l, 4, dict(score="sigmoid", renorm=True, n_group=8, topk_group=3,
                                       group_top=2, bias=bias))


@pytest.mark.parametrize("name", ["softmax", "sigmoid bias", "groups top2 bias"])
def test_route_scored_near_ties(torch, moe, name):
    """Neighbouring fp32 logits and biases: scores that differ in their last fp32 bits only are
    ordered as their 64-bit values are."""
    T, E, k = 128, 96, 8
    rng = np.random.default_rng(11)
    base = rng.standard_normal((T, 1)).astype(np.float32)
    steps = rng.integers(-3, 4, (T, E)).astype(np.float32)
    l = (base + steps * np.spacing(np.abs(base))).astype(np.float32)
    rule = dict(RULES[name])
    if "bias" in rule:
        rule["bias"] = (0.25 + rng.integers(-2, 3, E) * 2.0 ** -25).astype(np.float32)
    check_route(torch, moe, l, k, rule)


def test_route_scored_non_finite_rows(torch, moe):
    T, E, k = 9, 40, 4
    rng = np.random.default_rng(2)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[1, 39], l[4, 0], l[7, 20] = np.nan, np.inf, -np.inf
    ids, w, counts, offs, perm, inv, status = run_route(torch, moe, l, k, score="sigmoid")
    assert status == moe.ERR_NONFINITE
    rid, _ = ref.route(np.nan_to_num(l, nan=0, posinf=0, neginf=0), k, "sigmoid", 1, 1, 1, True, 1.0,
                       None)
    for t in (1, 4, 7):
        rid[t] = np.arange(k)
        assert np.array_equal(w[t], np.full(k, 0.25, np.float32))
    assert np.array_equal(ids, rid)
    assert np.array_equal(counts, ref.group(rid, E)[0])
    bias = np.zeros(E, np.float32)
    bias[3] = np.nan
    ids, _, _, _, _, _, status = run_route(torch, moe, np.zeros((2, E), np.float32), k, bias=bias)
    assert status == moe.ERR_NONFINITE and np.array_equal(ids, np.tile(np.arange(k), (2, 1)))


# ------------------------------------------------------------------ quantiser


def run_quantize(torch, moe, x, ldx=None, ldq=None, extra_rows=0):
    """x: torch tensor on the device [T][K] (a view with stride ldx)."""
    T, K = x.shape
    ldx = x.stride(0) if ldx is None else ldx
    ldq = -(-K // 16) * 16 if ldq is None else ldq
    q = torch.full((T, ldq), 0xAB, dtype=torch.uint8, device="cuda")
    lds = T + extra_rows
    s = torch.full((ref.blocks(K), lds), -3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.scaled_quantize(x.data_ptr(), moe.dtype_of(x), T, K, ldx, q.data_ptr(), ldq, s.data_ptr(),
                        lds, status.data_ptr(), _stream(torch))
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("dtype", list(EPS))
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (1, 128, 0), (3, 2560, 0), (5, 130, 0), (7, 127, 3),
                                     (66, 300, 4), (129, 641, 1), (4, 4096, 8)])
def test_quantize_bits(torch, moe, dtype, T, K, pad):
    rng = np.random.default_rng(T * 31 + K)
    x = rng.standard_normal((T, K + pad)) * np.exp(3 * rng.standard_normal((T, 1)))
    x[:, ::7] *= 20
    xd = _dev(torch, x).to(getattr(torch, dtype))[:, :K]
    q, s, status = run_quantize(torch, moe, xd, ldx=K + pad, ldq=-(-K // 16) * 16 + 32, extra_rows=3)
    rq, rs = ref.quantize(xd.double().cpu().numpy())
    # a few of these values pass the largest fp16: their blocks are reported
    assert status == (0 if bool(torch.isfinite(xd).all()) else moe.ERR_NONFINITE)
    assert np.array_equal(q[:, :K], rq) and np.array_equal(s[:, :T], rs)
    assert (q[:, K:] == 0xAB).all() and (s[:, T:] == -3.0).all()      # left as they were


def test_quantize_ties_zeros_and_extremes(torch, moe):
    """Quotients exactly halfway between e4m3 values, all-zero blocks, subnormal scales, the
    largest and smallest magnitudes."""
    rows = [np.concatenate([[448.0], ref._MID, [0.0]])[:128], np.zeros(128),
            np.full(128, 1e-45), np.full(128, -3e-42) * (1 + np.arange(128) % 3),
            np.linspace(-3.4e38, 3.4e38, 128), np.concatenate([[1e-36], np.full(127, 1e-44)]),
            -np.concatenate([[448.0 * 2 ** -9], ref._MID * 2.0 ** -9, [0.0]])[:128]]
    x = np.stack(rows).astype(np.float32)
    q, s, status = run_quantize(torch, moe, _dev(torch, x))
    rq, rs = ref.quantize(x)
    assert status == 0
    assert np.array_equal(s, rs)
    assert np.array_equal(ref.E4M3[q], ref.E4M3[rq])
    rng = np.random.default_rng(3)
    x = np.ldexp(rng.integers(-64, 65, (400, 256)).astype(np.float32), rng.integers(-20, 20, (400, 1)))
    q, s, _ = run_quantize(torch, moe, _dev(torch, x.astype(np.float32)))
    rq, rs = ref.quantize(x)
    assert np.array_equal(s, rs) and np.array_equal(ref.E4M3[q], ref.E4M3[rq])


def test_quantize_non_finite_blocks(torch, moe):
    x = np.random.default_rng(0).standard_normal((6, 384)).astype(np.float32)
    x[0, 5], x[2, 200], x[5, 383] = np.nan, np.inf, -np.inf
    q, s, status = run_quantize(torch, moe, _dev(torch, x))
    rq, rs = ref.quantize(x)
    assert status == moe.ERR_NONFINITE
    assert np.array_equal(q, rq) and np.array_equal(s, rs)
    assert s[0, 0] == 0 and s[1, 2] == 0 and s[2, 5] == 0 and (q[0, :128] == 0).all()


# ------------------------------------------------------------------ product


@pytest.mark.parametrize("dtype", list(EPS))
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 128), (1, 1280, 2560), (2, 130, 64), (7, 33, 300),
                                   (8, 257, 1000), (9, 16, 16), (16, 300, 128), (17, 128, 130),
                                   (64, 640, 2560), (127, 129, 257), (128, 256, 384), (129, 513, 500),
                                   (300, 100, 1296), (777, 1001, 144), (40, 2560, 4096),
                                   (1, 520, 8192), (513, 700, 640)])
def test_matmul(torch, moe, dtype, M, N, K):
    rng = np.random.default_rng(M * 131 + N * 17 + K)
    lda, ldb, ldas, ldo = -(-K // 16) * 16 + 16, -(-K // 16) * 16 + 32, M + 3, N + 5
    # bytes past column K are NaN codes, scales past row M NaN: neither may be used
    a, b = np.full((M, lda), 0x7F, np.uint8), np.full((N, ldb), 0xFF, np.uint8)
    a[:, :K] = ref.encode(np.clip(rng.standard_normal((M, K)) * 130, -448, 448))
    b[:, :K] = ref.encode(np.clip(rng.standard_normal((N, K)) * 130, -448, 448))
    sa = np.full((ref.blocks(K), ldas), np.nan, np.float32)
    sa[:, :M] = np.exp(rng.standard_normal((ref.blocks(K), M))) * 1e-2
    sb = (np.exp(rng.standard_normal((ref.blocks(N), ref.blocks(K)))) * 1e-3).astype(np.float32)
    ad, bd, sad, sbd = (_dev(torch, v) for v in (a, b, sa, sb))
    out = torch.full((M, ldo), -9.0, dtype=getattr(torch, dtype), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nb = moe.scaled_matmul_workspace_size(M, N, K)
    ws = torch.full((max(nb, 1),), 255, dtype=torch.uint8, device="cuda")

    def call():
        moe.scaled_matmul(ad.data_ptr(), lda, sad.data_ptr(), ldas, M, K, bd.data_ptr(), ldb,
                          sbd.data_ptr(), N, out.data_ptr(), moe.dtype_of(out), ldo,
                          status.data_ptr(), ws.data_ptr(), nb, _stream(torch))
        torch.cuda.synchronize()
        return out.clone()

    first = call()
    got = first.double().cpu().numpy()
    want, mag = ref.matmul(ref.wide_act(a[:, :K], sa[:, :M]), ref.wide_weight(b[:, :K], sb))
    assert int(status.item()) == 0
    err = np.abs(got[:, :N] - want)
    assert (err <= mag * ref.product_error(ref.blocks(K)) + np.abs(want) * EPS[dtype] +
            2.0 ** -25).all(), (err / mag).max()
    assert (got[:, N:] == -9.0).all()
    assert torch.equal(first.view(torch.uint8), call().view(torch.uint8))       # repeats bit for bit


def test_matmul_nan_and_zero_scales(torch, moe):
    """A NaN code reaches its row or column and no other; zero scales give zeros."""
    for M in (3, 40):
        N, K = 70, 256
        rng = np.random.default_rng(M)
        a = ref.encode(rng.standard_normal((M, K)) * 100)
        b = ref.encode(rng.standard_normal((N, K)) * 100)
        a[1, 130], b[5, 7] = 0x7F, 0xFF
        sa = np.ones((2, M), np.float32)
        sa[:, 2] = 0.0
        sb = np.ones((1, 2), np.float32)
        ad, bd, sad, sbd = (_dev(torch, v) for v in (a, b, sa, sb))
        out = torch.zeros(M, N, device="cuda")
        moe.scaled_matmul(ad.data_ptr(), K, sad.data_ptr(), M, M, K, bd.data_ptr(), K, sbd.data_ptr(),
                          N, out.data_ptr(), 0, N, None, None, 0, _stream(torch))
        got = out.cpu().numpy()
        want = np.zeros((M, N), bool)
        want[1], want[:, 5] = True, True
        assert np.array_equal(np.isnan(got), want)
        assert (got[2][~want[2]] == 0).all()


# ------------------------------------------------------------------ experts


def make_layer(torch, moe, rng, E, H, F, k, shared, T):
    W = {"shared": shared}
    for name, rows, cols in (("gate", F, H), ("up", F, H), ("down", H, F)):
        W[name] = ref.random_weights(rng, E + int(shared), rows, cols)
    t = [_dev(torch, W[n][i]) for n in ("gate", "up", "down") for i in (0, 1)]
    return W, moe.ScaledExperts(*t, T, k, shared=shared)


def run_experts(torch, layer, x, ids, w, gate, out_dtype):
    E = layer.n_experts
    counts, offs, perm, inv = ref.group(ids, E)
    layer.ws.fill_(0xA5)
    out = torch.full(x.shape, float("nan"), dtype=out_dtype, device="cuda")
    layer.forward(x, _dev(torch, ids), _dev(torch, w), _dev(torch, offs), _dev(torch, perm),
                  _dev(torch, inv), gate=None if gate is None else _dev(torch, gate), out=out)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("xt,ot", [("bfloat16", "bfloat16"), ("float32", "float32"),
                                   ("float16", "float16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("T,E,k,H,F,shared", [
    (1, 8, 2, 256, 128, False), (1, 6, 6, 144, 48, True), (2, 16, 4, 512, 640, True),
    (3, 40, 5, 384, 144, True), (8, 5, 3, 272, 272, False), (9, 8, 2, 256, 128, False),
    (16, 4, 4, 400, 80, True), (33, 24, 3, 144, 400, True), (150, 3, 2, 640, 256, True),
    (130, 64, 1, 256, 16, False), (300, 2, 1, 16, 128, True),
    (600, 3, 2, 272, 144, True), (700, 4, 1, 128, 656, False)])
def test_experts(torch, moe, xt, ot, T, E, k, H, F, shared):
    rng = np.random.default_rng(T * 1009 + E * 31 + H + F)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, shared, T)
    x = rng.standard_normal((T, H))
    x[:, ::50] *= 20
    xd = _dev(torch, x).to(getattr(torch, xt))
    ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    gate = rng.random(T).astype(np.float32) if shared and T % 2 else None
    out = run_experts(torch, layer, xd, ids, w, gate, getattr(torch, ot))
    assert layer.status() == 0
    want, tol, half = ref.experts(xd.double().cpu().numpy(), ids, w, gate, W)
    if T > 4 and ot != "float32":
        tol = tol + half
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol + np.abs(want) * EPS[ot] + 2.0 ** -25).all(), (err / tol).max()
    again = run_experts(torch, layer, xd, ids, w, gate, getattr(torch, ot))
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("T", [1, 7, 20])
def test_experts_same_expert_twice(torch, moe, T):
    """An id that a token names twice counts with both weights."""
    E, k, H, F = 6, 3, 256, 128
    rng = np.random.default_rng(T)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, False, T)
    x = rng.standard_normal((T, H)).astype(np.float32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[0] = 2
    w = rng.random((T, k)).astype(np.float32)
    out = run_experts(torch, layer, _dev(torch, x), ids, w, None, torch.float32)
    want, tol, half = ref.experts(x, ids, w, None, W)
    assert layer.status() == 0
    assert (np.abs(out.cpu().numpy() - want) <= tol + np.abs(want) * 2.0 ** -24).all()


@pytest.mark.parametrize("T", [4, 40])
def test_experts_non_finite_and_zero_tokens(torch, moe, T):
    """A block of x that is not finite is taken as zeros and reported; other tokens keep their
    bits; a token of zeros gives zeros."""
    E, k, H, F = 8, 2, 384, 128
    rng = np.random.default_rng(T)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, True, T)
    x = rng.standard_normal((T, H)).astype(np.float32)
    x[2] = 0.0
    ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    clean = run_experts(torch, layer, _dev(torch, x), ids, w, None, torch.float32).cpu().numpy()
    assert layer.status() == 0
    assert (clean[2] == 0).all()
    bad = x.copy()
    bad[1, 200] = np.inf
    got = run_experts(torch, layer, _dev(torch, bad), ids, w, None, torch.float32).cpu().numpy()
    assert layer.status() == moe.ERR_NONFINITE
    zeroed = x.copy()
    zeroed[1, 128:256] = 0
    same = run_experts(torch, layer, _dev(torch, zeroed), ids, w, None, torch.float32).cpu().numpy()
    assert np.array_equal(got, same)
    others = np.arange(T) != 1
    assert np.array_equal(got[others], clean[others])


@pytest.mark.parametrize("T", [3, 40])
def test_experts_out_of_range_ids_are_skipped(torch, moe, T):
    """An id or a slot that no router wrote is reported and takes no part; nothing is read past
    the experts or the slots."""
    E, k, H, F = 6, 2, 256, 128
    rng = np.random.default_rng(T)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, False, T)
    x = _dev(torch, rng.standard_normal((T, H)).astype(np.float32))
    ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    counts, offs, perm, inv = ref.group(ids, E)
    bad_ids, bad_inv = ids.copy(), inv.copy()
    bad_ids[1, 0] = E + 3
    bad_inv[2 * k + 1] = T * k + 5
    out = torch.zeros(T, H, device="cuda")
    layer.forward(x, _dev(torch, bad_ids), _dev(torch, w), _dev(torch, offs), _dev(torch, perm),
                  _dev(torch, bad_inv if T > 4 else inv), out=out)
    assert layer.status() == moe.ERR_BOUNDS
    w2 = w.copy()
    w2[1, 0] = 0
    if T > 4:
        w2[2, 1] = 0
    want, tol, half = ref.experts(x.cpu().numpy(), ids, w2, None, W)
    # what is left out differs from what a zero weight adds by the rounding of a sum at most
    err = np.abs(out.cpu().numpy() - want)
    assert (err <= tol + np.abs(want) * 2.0 ** -24).all()


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("T", [1, 6, 37, 200])
def test_route_then_experts_eager_captured_and_on_another_stream(torch, moe, T):
    """The router and the experts as a decoder layer runs them, against the plain forms; the same
    calls replayed from a CUDA graph on new inputs, and run on a side stream, give the same bits."""
    E, k, H, F = 24, 4, 384, 144
    rng = np.random.default_rng(T)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, True, T)
    bias = _dev(torch, (0.1 * rng.standard_normal(E)).astype(np.float32))
    layer.rule = moe.RouteRule(moe.SCORE_SIGMOID, 4, 2, 2, True, 2.5, bias.data_ptr())
    xs = [_dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16) for _ in range(2)]
    ls = [_dev(torch, (2 * rng.standard_normal((T, E))).astype(np.float32)) for _ in range(2)]
    gate = _dev(torch, rng.random(T).astype(np.float32))
    eager = [layer(x, l, gate=gate).clone() for x, l in zip(xs, ls)]
    assert layer.status() == 0
    for x, l, o in zip(xs, ls, eager):
        ids, w = ref.route(l.cpu().numpy(), k, "sigmoid", 4, 2, 2, True, 2.5, bias.cpu().numpy())
        assert np.array_equal(layer.route(l)[0].cpu().numpy(), ids)
        want, tol, half = ref.experts(x.double().cpu().numpy(), ids, w.astype(np.float32),
                                gate.cpu().numpy(), W)
        # the routing weights carry half an fp32 step, like a rounding of y
        tol = tol + half * (T > 4)
        err = np.abs(o.double().cpu().numpy() - want)
        assert (err <= tol + np.abs(want) * EPS["bfloat16"]).all()
    x, l = xs[0].clone(), ls[0].clone()
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, l, gate=gate, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, l, gate=gate, out=out)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        l.copy_(ls[i])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
    assert layer.status() == 0


# ------------------------------------------------------------------ calls that share or grow


@pytest.mark.parametrize("dtype", list(EPS))
@pytest.mark.parametrize("M,N,K", [(2000, 1301, 144), (3001, 2003, 130), (2304, 2064, 272)])
def test_matmul_of_more_tiles_than_run_at_once(torch, moe, dtype, M, N, K):
    """Wide tiles: one per CTA, and several, with rows of any alignment and with aligned ones."""
    ldo = N + (5 if N % 16 else 0)
    rng = np.random.default_rng(M + N + K)
    kp = -(-K // 16) * 16
    a, b = np.full((M, kp), 0x7F, np.uint8), np.full((N, kp), 0xFF, np.uint8)
    a[:, :K] = ref.encode(np.clip(rng.standard_normal((M, K)) * 130, -448, 448))
    b[:, :K] = ref.encode(np.clip(rng.standard_normal((N, K)) * 130, -448, 448))
    sa = (np.exp(rng.standard_normal((ref.blocks(K), M))) * 1e-2).astype(np.float32)
    sb = (np.exp(rng.standard_normal((ref.blocks(N), ref.blocks(K)))) * 1e-3).astype(np.float32)
    ad, bd, sad, sbd = (_dev(torch, v) for v in (a, b, sa, sb))
    out = torch.full((M, ldo), -9.0, dtype=getattr(torch, dtype), device="cuda")
    moe.scaled_matmul(ad.data_ptr(), kp, sad.data_ptr(), M, M, K, bd.data_ptr(), kp, sbd.data_ptr(),
                      N, out.data_ptr(), moe.dtype_of(out), ldo, None, None, 0, _stream(torch))
    got = out.double().cpu().numpy()
    want, mag = ref.matmul(ref.wide_act(a[:, :K], sa), ref.wide_weight(b[:, :K], sb))
    err = np.abs(got[:, :N] - want)
    assert (err <= mag * ref.product_error(ref.blocks(K)) + np.abs(want) * EPS[dtype] +
            2.0 ** -25).all(), (err / mag).max()
    assert (got[:, N:] == -9.0).all()


@pytest.mark.parametrize("M", [5, 200])
def test_product_and_quantiser_past_32_bit_offsets(torch, moe, M):
    """Rows so far apart that the last ones lie past 2^32 bytes; what lies between them is left."""
    pitch, K, N = (1 << 32) // (M - 1) // 16 * 16 + 4096, 272, 48
    assert (M - 1) * pitch > 1 << 32
    rng = np.random.default_rng(M)
    x = _dev(torch, rng.standard_normal((M, K)).astype(np.float32))
    store = torch.full((M * pitch,), 0x55, dtype=torch.uint8, device="cuda")
    q = store.view(M, pitch)
    s = torch.empty((ref.blocks(K), M), device="cuda")
    moe.scaled_quantize(x.data_ptr(), 0, M, K, K, q.data_ptr(), pitch, s.data_ptr(), M, None,
                        _stream(torch))
    rq, rs = ref.quantize(x.cpu().numpy())
    assert np.array_equal(q[:, :K].cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    assert (q[:, K:K + 64] == 0x55).all()
    b = ref.encode(rng.standard_normal((N, K)) * 100)
    sb = np.full((ref.blocks(N), ref.blocks(K)), 1e-2, np.float32)
    bd, sbd = _dev(torch, b), _dev(torch, sb)
    near, out = torch.empty((M, N), device="cuda"), None
    moe.scaled_matmul(q.data_ptr(), pitch, s.data_ptr(), M, M, K, bd.data_ptr(), K, sbd.data_ptr(),
                      N, near.data_ptr(), 0, N, None, None, 0, _stream(torch))
    want, mag = ref.matmul(ref.wide_act(rq, rs), ref.wide_weight(b, sb))
    assert (np.abs(near.cpu().numpy() - want) <= mag * ref.product_error(ref.blocks(K)) +
            np.abs(want) * EPS["float32"] + 2.0 ** -25).all()
    # the same activations close together, the output's rows far apart
    qd, ldo = _dev(torch, rq), pitch // 4
    store.fill_(0x55)
    out = store.view(torch.float32).view(M, ldo)
    moe.scaled_matmul(qd.data_ptr(), K, s.data_ptr(), M, M, K, bd.data_ptr(), K, sbd.data_ptr(), N,
                      out.data_ptr(), 0, ldo, None, None, 0, _stream(torch))
    assert torch.equal(out[:, :N], near)
    assert (out[:, N:N + 64].contiguous().view(torch.uint8) == 0x55).all()


def _layer_inputs(torch, moe, T, seed):
    E, k, H, F = 24, 4, 384, 144
    rng = np.random.default_rng(seed)
    _, layer = make_layer(torch, moe, rng, E, H, F, k, True, T)
    x = _dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16)
    l = _dev(torch, (2 * rng.standard_normal((T, E))).astype(np.float32))
    return layer, x, l


@pytest.mark.parametrize("T", [1, 5, 50])
def test_two_layers_at_once_on_two_streams(torch, moe, T):
    """Layers share nothing: each with its own workspace, their calls overlap."""
    a, b = _layer_inputs(torch, moe, T, 1), _layer_inputs(torch, moe, T, 2)
    want = [l(x, lg) for l, x, lg in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, (l, x, lg) in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(l(x, lg))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])
    assert a[0].status() == 0 and b[0].status() == 0


def test_graphs_that_share_a_workspace(torch, moe):
    """Graphs of one layer at 1, 5 and 50 tokens use one workspace; replayed in any order on one
    stream, with eager calls between, each gives its own result.  The output may be x itself."""
    layer, x, l = _layer_inputs(torch, moe, 50, 3)
    sizes = (1, 5, 50)
    want = {T: layer(x[:T], l[:T]).clone() for T in sizes}
    graphs, buf = {}, {T: x[:T].clone() for T in sizes}
    torch.cuda.synchronize()
    for T in sizes:
        graphs[T] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[T]):
            layer(buf[T], l[:T], out=buf[T])
    for T in (50, 1, 5, 1, 50, 50, 5):
        buf[T].copy_(x[:T])
        graphs[T].replay()
        assert torch.equal(layer(x[:7], l[:7]), layer(x[:7], l[:7]))
        assert torch.equal(buf[T], want[T])
    assert layer.status() == 0


FIRST_CALL = """
import sys, torch
sys.path[:0] = {path!r}
from expert_ffn_token_b200 import moe
import test_gpu_scaled as t
for T in (1, 5, 50):
    layer, x, l = t._layer_inputs(torch, moe, T, T)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, l, out=out)
    g.replay()
    assert torch.equal(out, layer(x, l)) and layer.status() == 0
print("same")
"""


def test_first_call_of_a_process_may_be_captured(torch, moe):
    """Nothing is loaded, allocated or waited for on a first call that a capture forbids."""
    import os
    import subprocess
    import sys

    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(path=[os.path.dirname(here), here])
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


# ------------------------------------------------------------------ waits that run out


@pytest.fixture
def short_waits(moe):
    """A limit far below what the kernels' hand-overs take, and the default again afterwards."""
    moe.scaled_set_wait_limit(1)
    yield
    moe.scaled_set_wait_limit(2_000_000_000)


def _product(torch, moe, M, N, K):
    rng = np.random.default_rng(M + N)
    a = ref.encode(np.clip(rng.standard_normal((M, K)) * 130, -448, 448))
    b = ref.encode(np.clip(rng.standard_normal((N, K)) * 130, -448, 448))
    t = [_dev(torch, v) for v in (a, np.full((ref.blocks(K), M), 1e-2, np.float32), b,
                                  np.full((ref.blocks(N), ref.blocks(K)), 1e-3, np.float32))]
    out = torch.zeros((M, N), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        moe.scaled_matmul(t[0].data_ptr(), K, t[1].data_ptr(), M, M, K, t[2].data_ptr(), K,
                          t[3].data_ptr(), N, out.data_ptr(), 0, N, status.data_ptr(), None, 0,
                          _stream(torch))
        torch.cuda.synchronize()
        return moe.read_status(status.data_ptr(), _stream(torch))

    return call, out


@pytest.mark.parametrize("M,N,K", [(300, 512, 4096), (2048, 2560, 4096)])
def test_matmul_wait_times_out_and_next_call_is_clean(torch, moe, short_waits, M, N, K):
    """The product's kernels (tiles of 128 and of 256 weight rows) report a wait that runs out, end,
    and leave nothing behind: the next call's result is the bits of an undisturbed one."""
    call, out = _product(torch, moe, M, N, K)
    assert call() == moe.ERR_TIMEOUT
    moe.scaled_set_wait_limit(2_000_000_000)
    assert call() == 0
    first = out.clone()
    moe.scaled_set_wait_limit(1)
    assert [call() for _ in range(5)] == [moe.ERR_TIMEOUT] * 5
    moe.scaled_set_wait_limit(2_000_000_000)
    out.zero_()
    assert call() == 0 and torch.equal(out, first)


@pytest.mark.parametrize("T", [60, 700])
def test_experts_wait_times_out_and_next_call_is_clean(torch, moe, short_waits, T):
    """Likewise for the experts' gate/up and down, whose epilogue warps also wait for one another."""
    E, k, H, F = 8, 3, 2048, 640
    rng = np.random.default_rng(T)
    _, layer = make_layer(torch, moe, rng, E, H, F, k, True, T)
    x = _dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16)
    l = _dev(torch, (2 * rng.standard_normal((T, E))).astype(np.float32))
    layer(x, l)
    assert layer.status() == moe.ERR_TIMEOUT
    moe.scaled_set_wait_limit(2_000_000_000)
    first = layer(x, l)
    assert layer.status() == 0
    for _ in range(5):
        moe.scaled_set_wait_limit(1)
        layer(x, l)
        assert layer.status() == moe.ERR_TIMEOUT
        moe.scaled_set_wait_limit(2_000_000_000)
        assert torch.equal(layer(x, l), first)
        assert layer.status() == 0


# ------------------------------------------------------------------ what y and h are held in


@pytest.mark.parametrize("T,E,k,H,F,shared", [(5, 16, 4, 512, 640, True), (40, 24, 8, 400, 272, False),
                                              (200, 12, 6, 640, 256, True)])
def test_experts_fp16_output_is_rounded_once(torch, moe, T, E, k, H, F, shared):
    """With an fp16 output y is not held in fp16: the sum of k outputs that nearly cancel keeps the
    accuracy of fp32 sums.  tol is the fp32 arithmetic's, EPS the output's own rounding."""
    rng = np.random.default_rng(T + F)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, shared, T)
    x = rng.standard_normal((T, H))
    xd = _dev(torch, x).to(torch.float16)
    ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.standard_normal((T, k)).astype(np.float32)
    out = run_experts(torch, layer, xd, ids, w, None, torch.float16)
    want, tol, _ = ref.experts(xd.double().cpu().numpy(), ids, w, None, W)
    assert layer.status() == 0
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol + np.abs(want) * EPS["float16"] + 2.0 ** -25).all()


def magnitudes(x, ids, w, gate, W):
    """The sum of |weight * y| over a token's experts [T][H] in 64 bits."""
    T, E = x.shape[0], W["gate"][0].shape[0] - int(W["shared"])
    xq = ref.wide_act(*ref.quantize(x))
    c = np.zeros((T, E + int(W["shared"])))
    np.add.at(c, (np.arange(T)[:, None], ids), w.astype(np.float64))
    if W["shared"]:
        c[:, E] = 1.0 if gate is None else gate
    out = np.zeros((T, W["down"][0].shape[1]))
    for e in range(c.shape[1]):
        m = {n: ref.wide_weight(W[n][0][e], W[n][1][e]) for n in ("gate", "up", "down")}
        g, u = xq @ m["gate"].T, xq @ m["up"].T
        y = ref.wide_act(*ref.quantize(g / (1 + np.exp(-g)) * u)) @ m["down"].T
        out += np.abs(c[:, e:e + 1] * y)
    return out


@pytest.mark.parametrize("unused", [1.0, 2.0 ** 20])
@pytest.mark.parametrize("T,E,k,H,F", [(5, 8, 3, 400, 640), (150, 6, 2, 640, 384)])
def test_experts_bf16_output_with_unused_scales(torch, moe, T, E, k, H, F, unused):
    """A block of zero weights may be stored with any scale (1 instead of 0, say); what the other
    blocks give keeps its accuracy.  y in fp16 may be off by 2^-11 of it, or by 2^-25 times its power of
    two, which is at most 2^-14 of the largest of 32 columns."""
    rng = np.random.default_rng(T + F)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, False, T)
    codes, scales = W["down"]
    codes[:, :, 128:256] = 0
    scales *= 2.0 ** -12                        # weights of 2^-20 and so
    scales[:, :, 1] = unused
    W["down"] = codes, scales
    layer.tensors[2].copy_(_dev(torch, codes))
    layer.tensors[5].copy_(_dev(torch, scales))
    xd = _dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16)
    ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    x = xd.double().cpu().numpy()
    out = run_experts(torch, layer, xd, ids, w, None, torch.bfloat16)
    want, tol, _ = ref.experts(x, ids, w, None, W)
    mag = magnitudes(x, ids, w, None, W)
    top = np.repeat(np.stack([mag[:, i:i + 32].max(1) for i in range(0, H, 32)], 1), 32, 1)[:, :H]
    assert layer.status() == 0
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol + mag * 2.0 ** -11 + top * 2.0 ** -39 + np.abs(want) * EPS["bfloat16"]).all()


def test_experts_bf16_output_of_extreme_magnitudes(torch, moe):
    """y from 2^-90 to near the largest fp32 (below, a product of two scales is no normal number): the
    power of two follows."""
    T, E, k, H, F = 12, 4, 1, 256, 128
    rng = np.random.default_rng(0)
    W, layer = make_layer(torch, moe, rng, E, H, F, k, False, T)
    xd = _dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16)
    x = xd.double().cpu().numpy()
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    w = np.ones((T, 1), np.float32)
    base = W["down"][1].copy()
    for power in (-90, -30, -14, 0, 14, 60, 118):
        W["down"] = W["down"][0], (base * 2.0 ** power).astype(np.float32)
        layer.tensors[5].copy_(_dev(torch, W["down"][1]))
        out = run_experts(torch, layer, xd, ids, w, None, torch.bfloat16)
        want, tol, _ = ref.experts(x, ids, w, None, W)
        top = np.abs(want).max(1, keepdims=True)
        assert layer.status() == 0
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= tol + np.abs(want) * (2.0 ** -11 + EPS["bfloat16"]) + top * 2.0 ** -39).all(), power


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [0, 40, -120])
@pytest.mark.parametrize("T", [1, 3, 5, 20, 140])
def test_experts_h_halfway_between_e4m3_values(torch, moe, T, power, sign):
    """h exactly halfway between each two e4m3 values goes to the even one, whatever the batch size:
    g is 128, whose silu is 128; u is 448 w1 + 28 w2 = 448 m for the midpoint m; h is 448 * 128 m, of
    which the largest, m = 448, makes the scale 448 * 128; the down matrix hands h^ out."""
    E, H, F = 2, 256, 128
    m = np.concatenate([sign * ref._MID, [448.0, 0.0]])
    low = np.concatenate([ref._POS[:-1], [448.0, 0.0]])
    step = np.concatenate([8 * np.diff(ref._POS), [0.0, 0.0]])
    x = np.zeros((T, H), np.float32)
    x[:, :3] = 448, 28, 64
    W = {"shared": False}
    gate, up, down = np.zeros((E, F, H)), np.zeros((E, F, H)), np.zeros((E, H, F))
    gate[:, :, 2] = 2
    up[:, :, 0], up[:, :, 1] = np.sign(m) * low, np.sign(m) * step
    down[:, np.arange(F), np.arange(F)] = 1
    scale = {"gate": 1.0, "up": 2.0 ** power, "down": 2.0 ** -power}
    for name, v in (("gate", gate), ("up", up), ("down", down)):
        assert np.array_equal(ref.E4M3[ref.encode(v)], v)
        s = np.full((E, ref.blocks(v.shape[1]), ref.blocks(v.shape[2])), scale[name], np.float32)
        W[name] = ref.encode(v), s
    layer = moe.ScaledExperts(*(_dev(torch, W[n][i]) for n in ("gate", "up", "down") for i in (0, 1)),
                              T, 1)
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    out = run_experts(torch, layer, _dev(torch, x), ids, np.ones((T, 1), np.float32), None,
                      torch.float32).cpu().numpy()
    assert layer.status() == 0
    want = np.zeros(H)
    want[:F] = ref.E4M3[ref.encode(m)] * 448 * 128
    assert (out == want).all(), np.argwhere(out[0] != want).ravel()


@pytest.mark.parametrize("T", [1, 3, 5, 20])
def test_experts_h_of_very_negative_gates(torch, moe, T):
    """silu from -60 down to fp32's smallest normal results keeps its accuracy at every batch size: a
    block of such h is as accurate as any other, since its scale is its own.  Four fp32 exponentials
    and roundings are at most 2^-20 of h; where that crosses a midpoint, the neighbour is right."""
    E, H, F = 2, 256, 128
    rng = np.random.default_rng(T)
    for g in (-60.0, -79.0, -81.0, -83.0, -86.0, -87.5, -88.5, -90.0):
        u = rng.choice(ref._POS[64:100], F)
        x = np.zeros((T, H), np.float32)
        x[:, 0], x[:, 1] = 448, 64
        v = {"gate": np.zeros((E, F, H)), "up": np.zeros((E, F, H)), "down": np.zeros((E, H, F))}
        v["gate"][:, :, 1] = 1
        v["up"][:, :, 0] = u
        v["down"][:, np.arange(F), np.arange(F)] = 1
        scale = {"gate": g / 64, "up": 2.0 ** 60, "down": 2.0 ** 50}
        W = {n: (ref.encode(m), np.full((E, ref.blocks(m.shape[1]), ref.blocks(m.shape[2])), scale[n],
                                        np.float32)) for n, m in v.items()}
        layer = moe.ScaledExperts(*(_dev(torch, W[n][i]) for n in v for i in (0, 1)), T, 1)
        ids = (np.arange(T) % E).astype(np.int32)[:, None]
        out = run_experts(torch, layer, _dev(torch, x), ids, np.ones((T, 1), np.float32), None,
                          torch.float32).cpu().numpy().astype(np.float64)[:, :F]
        assert layer.status() == 0
        g32 = float(np.float32(64) * W["gate"][1][0, 0, 0])
        h = g32 / (1 + np.exp(-g32)) * 448 * u * 2.0 ** 60
        r = np.abs(h) / np.abs(h).max() * 448            # all of one block: the scale's error cancels
        lo, hi = (ref.E4M3[ref.encode(r * (1 + f * 2.0 ** -20))] for f in (-1, 1))
        s = np.abs(h).max() / 448 * 2.0 ** 50
        assert (-out >= lo * s * (1 - 2.0 ** -19)).all() and (-out <= hi * s * (1 + 2.0 ** -19)).all(), g


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (70, 512, 10), (9, 1000, 32), (40, 60, 6), (5, 1032, 8)])
@pytest.mark.parametrize("rule", [dict(), dict(n_group=4, topk_group=2, group_top=2)])
def test_route_scored_softmax_weights_are_rounded_once(torch, moe, T, E, k, rule):
    """Weights that are not renormalised are the 64-bit softmax, rounded to fp32 once (half a step; the
    64-bit arithmetic is off by less than 2^-40)."""
    rng = np.random.default_rng(T + E)
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    ids, w, *_, status = run_route(torch, moe, l, k, renorm=False, **rule)
    full = dict(n_group=1, topk_group=1, group_top=1)
    full.update(rule)
    rid, rw = ref.route(l, k, "softmax", renorm=False, scale=1.0, bias=None, **full)
    assert status == 0 and np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= (2.0 ** -24 + 2.0 ** -40) * rw).all()


@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (512, 10), (120, 5), (1000, 12)])
@pytest.mark.parametrize("mask", [-1e9, float(np.finfo(np.float32).min), -300.0])
@pytest.mark.parametrize("name", ["softmax bias", "sigmoid bias", "groups top1 bias", "groups top2 bias"])
def test_route_scored_masked_by_the_bias(torch, moe, name, mask, E, k):
    """Experts masked by a large negative bias, whole groups among them, leave near ties of the open
    ones to be decided as 64-bit values decide them; so do single experts with large biases."""
    T = 96
    rng = np.random.default_rng(E + k)
    rule = dict(RULES[name])
    bias = (0.25 + rng.integers(-2, 3, E) * 2.0 ** -25).astype(np.float32)
    per = E // 4
    bias[rng.permutation(E)[:E // 3]] = mask
    bias[:per] = mask                                   # a whole group
    bias[per + 2:2 * per] = mask                        # a group of at most two open experts
    bias[-per:-per + 3] = 1e6                           # and some that tie far above the scores
    rule["bias"] = bias
    base = rng.standard_normal((T, 1)).astype(np.float32)
    steps = rng.integers(-3, 4, (T, E)).astype(np.float32)
    l = (base + steps * np.spacing(np.abs(base))).astype(np.float32)
    l[T // 2:] = (2 * rng.standard_normal((T - T // 2, E))).astype(np.float32)
    check_route(torch, moe, l, k, rule)


def _random_layer(torch, moe, rng, E, H, F, k, shared, T):
    """Codes even over all finite e4m3 values, which are quick to draw."""
    W = {"shared": shared}
    n = E + int(shared)
    for name, rows, cols in (("gate", F, H), ("up", F, H), ("down", H, F)):
        q = rng.integers(0, 127, (n, rows, cols), dtype=np.uint8)
        q |= rng.integers(0, 2, q.shape, dtype=np.uint8) << 7
        s = np.exp(0.5 * rng.standard_normal((n, ref.blocks(rows), ref.blocks(cols))))
        W[name] = q, (s / (110 * cols ** 0.5)).astype(np.float32)
    t = [_dev(torch, W[m][i]) for m in ("gate", "up", "down") for i in (0, 1)]
    return W, moe.ScaledExperts(*t, T, k, shared=shared)


@pytest.mark.parametrize("E,k,H,F,shared,sizes", [
    (12, 10, 2560, 640, True, (1, 3, 5, 40, 300)), (256, 8, 256, 128, True, (2, 6, 70)),
    (2, 1, 7168, 2048, False, (1, 4, 20)), (1, 1, 16, 4096, False, (2, 9)), (3, 3, 4096, 16, True, (4, 5))])
def test_experts_of_whole_layers(torch, moe, E, k, H, F, shared, sizes):
    """Layers as large as those in use, long and thin ones, and many experts, at each batch size's
    kernels and with each output type."""
    rng = np.random.default_rng(H + F)
    W, layer = _random_layer(torch, moe, rng, E, H, F, k, shared, max(sizes))
    for T in sizes:
        xd = _dev(torch, rng.standard_normal((T, H))).to(torch.bfloat16)
        ids = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k].astype(np.int32)
        w = rng.random((T, k)).astype(np.float32)
        x = xd.double().cpu().numpy()
        want, tol, _ = ref.experts(x, ids, w, None, W)
        for dtype in EPS:
            out = run_experts(torch, layer, xd, ids, w, None, getattr(torch, dtype))
            allowed = tol + np.abs(want) * EPS[dtype] + 2.0 ** -25
            if T > 4 and dtype == "bfloat16":
                mag = magnitudes(x, ids, w, None, W)
                allowed += mag * 2.0 ** -11 + mag.max(1, keepdims=True) * 2.0 ** -39
            err = np.abs(out.double().cpu().numpy() - want)
            assert layer.status() == 0
            assert (err <= allowed).all(), (T, dtype, (err / allowed).max())


@pytest.mark.parametrize("dtype", list(EPS))
@pytest.mark.parametrize("T", [1, 3, 6, 140])
def test_experts_infinite_output_leaves_its_neighbours(torch, moe, T, dtype):
    """An output column that passes fp32 (a weight scale of 2^126) or is NaN (a NaN code) is that, and its
    neighbours are what they are without it."""
    E, H, F = 2, 64, 256
    rng = np.random.default_rng(T)
    W, layer = make_layer(torch, moe, rng, E, H, F, 1, False, T)
    codes, scales = W["down"]
    codes[:, :, 128:] = 0
    layer.tensors[2].copy_(_dev(torch, codes))
    xd = _dev(torch, rng.standard_normal((T, H))).to(getattr(torch, dtype))
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    w = np.ones((T, 1), np.float32)
    clean = run_experts(torch, layer, xd, ids, w, None, getattr(torch, dtype))
    # row 5 takes the largest h of the second block, 448 of its scale, times 448 * 2^126
    codes[:, 5, 128:], codes[:, 40, 200] = ref.encode(np.array([448.0])), 0x7F
    scales[:, :, 1] = 2.0 ** 126
    layer.tensors[2].copy_(_dev(torch, codes))
    layer.tensors[5].copy_(_dev(torch, scales))
    out = run_experts(torch, layer, xd, ids, w, None, getattr(torch, dtype))
    others = np.ones(H, bool)
    others[[5, 40]] = False
    keep = torch.from_numpy(np.flatnonzero(others)).cuda()
    assert layer.status() == 0
    # (the sum of 128 values of either sign that row 5 takes may by chance stay within fp32; then it
    # is a finite neighbour, 2^-39 of which the others may be off by)
    past = ~torch.isfinite(out[:, 5])
    assert past.double().mean() > 0.9 and torch.isnan(out[:, 40]).all()
    assert torch.isfinite(out[:, keep]).all()
    out, clean = out[past], clean[past]
    # the power of two may change with the neighbours gone, and with it subnormal fp16 values alone
    gap = (out[:, keep].double() - clean[:, keep].double()).abs()
    assert (gap <= clean[:, keep].double().abs() * 2 * EPS[dtype] * (dtype == "bfloat16") +
            clean.double().abs().amax() * 2.0 ** -38).all()
