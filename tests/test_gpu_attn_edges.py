"""The cache and attention calls at their edges: bounds that no work unit meets, numbers that are not finite, what a
pack's neighbours may change, waits that run out, a long sequence among many short ones.  Bounds of errors are those
that tests/test_gpu_attn.py derives; what a test adds to them stands in its docstring."""
import numpy as np
import pytest

import attn_reference as ref
from helpers import cuda, lib, to_np, torch
from test_gpu_attn import (append_case, bound, check_cache, check_decode, cu_of, decode_case, dev_cache, dtype, half_step,
                           lse_bound, rounded, run_decode, same_bits, split)

pytestmark = pytest.mark.gpu
BLOCK = ref.BLOCK


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch().cuda.is_available():
        pytest.skip("no CUDA device")
    yield


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert lib().bitnet_get_device_error() == lib().BITNET_OK


def ints(*x):
    return cuda(np.array(x, np.int32))


BAD_BOUNDS = [
    # tokens, bounds: no work unit looks at the pair that is wrong
    (2, [0, 1, 2, 3]),       # a unit for each token: the third sequence has none
    (2, [0, 1, 0, 1]),       # ... and the second goes backwards between two that are found
    (3, [-1, 0, 1, 2]),      # ... the first begins before row 0 and ends at it
    (4, [0, 1, 2, 2, 5]),
    (80, [0, 70, 10, 80]),   # units of 16 tokens: the second and third sequence begin at the same unit
    (300, [0, 140, 20, 300]),
]


@pytest.mark.parametrize("tokens,bounds", BAD_BOUNDS)
def test_bad_bounds_are_latched_by_every_packed_call(tokens, bounds):
    b, tt = lib(), torch()
    dim, hk, page, seqs = 64, 2, 16, len(bounds) - 1
    host = ref.Cache(seqs * 20, hk, page, dim)
    dev, table = dev_cache(host), cuda(np.arange(seqs * 20, dtype=np.int32).reshape(seqs, 20))
    x, cu, good = tt.ones((tokens, hk, dim), device="cuda"), ints(*bounds), ints(*[0] * seqs, tokens)
    zero = ints(*[0] * seqs)
    x16, out = x.half(), tt.empty((tokens, hk, dim), device="cuda")
    calls = {
        "append": lambda c: b.bitnet_kv_append(dev, x, x, x, c, zero, table, out),
        "gather": lambda c: b.bitnet_kv_gather(dev, c, table, out, tt.empty_like(out)),
        "prompt, queries": lambda c: b.bitnet_attn_prompt(x16, x16, x16, c, good, out),
        "prompt, keys": lambda c: b.bitnet_attn_prompt(x16, x16, x16, good, c, out),
    }
    for name, call in calls.items():
        call(cu)
        assert b.bitnet_get_device_error() == b.BITNET_ERR_VALUE, name
        call(good)
        assert b.bitnet_get_device_error() == b.BITNET_OK, name


@pytest.mark.parametrize("wrong", [0, 1, 700, 2998, 2999])
def test_one_bad_bound_among_many_sequences(wrong):
    """3000 sequences of one token, one of them backwards; then a negative length of a sequence without new tokens."""
    b, tt = lib(), torch()
    dim, seqs = 64, 3000
    dev = dev_cache(ref.Cache(seqs, 1, 16, dim))
    x, out = tt.ones((seqs, 1, dim), device="cuda"), tt.empty((seqs, 1, dim), device="cuda")
    table, old = tt.arange(seqs, dtype=tt.int32, device="cuda").view(-1, 1), tt.zeros(seqs, dtype=tt.int32, device="cuda")
    cu = np.arange(seqs + 1, dtype=np.int32)
    bad = cu.copy()
    bad[wrong + 1] = bad[wrong] - 1 if wrong else -1
    for c, o, want in ((bad, old, b.BITNET_ERR_VALUE), (cu, old, b.BITNET_OK)):
        b.bitnet_kv_append(dev, x, x, x, cuda(c), o, table, out)
        assert b.bitnet_get_device_error() == want
    empty = cu.copy()
    empty[wrong + 1:] -= 1   # no new token of that sequence
    negative = old.clone()
    negative[wrong] = -1
    for o, want in ((negative, b.BITNET_ERR_VALUE), (old, b.BITNET_OK)):
        b.bitnet_kv_append(dev, x[1:], x[1:], x[1:], cuda(empty), o, table, out[1:])
        assert b.bitnet_get_device_error() == want


def prompt(q, k, v, cu_q, cu_k, causal=True, scale=None, out=None):
    """(out, lse) of a call on device tensors; out fp32 unless a dtype is given."""
    b, tt = lib(), torch()
    o = tt.full(q.shape, 9.0, dtype=out or tt.float32, device="cuda")
    lse = tt.full(q.shape[:2], 9.0, device="cuda")
    b.bitnet_attn_prompt(q, k, v, ints(*cu_q), ints(*cu_k), o, causal=causal, scale=scale, lse=lse)
    return o, lse


@pytest.mark.parametrize("dim,t,causal", [(64, "f16", True), (64, "bf16", False), (128, "bf16", True), (128, "f16", False)])
def test_prompt_bits_do_not_depend_on_the_queries_packed_behind(dim, t, causal):
    """Rows behind a sequence's end in its last tile are the next sequence's queries: whatever those are (and NaN or
    infinite), the sequence's own rows keep their bits."""
    tt = torch()
    rng = np.random.default_rng(15)
    lens = [150, 106, 300]
    cu = cu_of(lens)
    q, k, v = (cuda(rng.normal(0, 1, (sum(lens), 4, dim)).astype(np.float32)).to(dtype(t)) for _ in range(3))
    want = prompt(q, k, v, cu, cu, causal)
    for i in range(3):
        own = slice(int(cu[i]), int(cu[i + 1]))
        for other in (200 * tt.randn_like(q), tt.full_like(q, float("nan")), tt.full_like(q, float("inf"))):
            other[own] = q[own]
            for a, w in zip(prompt(other, k, v, cu, cu, causal), want):
                assert tt.equal(a[own], w[own]), f"sequence {i}"


def check_rows(got, lse, q, k, v, seen, t, good):
    """Rows x heads of `good` are within the bounds, of the sequences' own formula on q, k, v (numpy, finite); the others
    are NaN in every element, and so are their lse."""
    dim = q.shape[2]
    o, z, mag, size, _ = ref.attend(q, k, v, dim ** -0.5, seen)
    g, l = to_np(got.double()), to_np(lse.double())
    assert np.isnan(g[~good]).all() and np.isnan(l[~good]).all()
    err = np.abs(g - o)
    assert np.all((err <= bound(mag, size, o, k.shape[0], dim, half_step(t), "f32"))[good])
    some = good & np.isfinite(z)
    assert np.all((np.abs(l - np.where(some, z, 0)) <= lse_bound(z, size, k.shape[0], dim))[some])
    assert np.all(g[good & ~some] == 0) and np.all(np.isneginf(l[good & ~some]))


NAN_PROMPTS = [(64, "f16", 300, True), (64, "bf16", 300, False), (128, "bf16", 300, True), (128, "f16", 300, False),
               (128, "bf16", 3, True)]


@pytest.mark.parametrize("dim,t,n,causal", NAN_PROMPTS)
def test_prompt_nan_in_a_query_makes_its_row_nan(dim, t, n, causal):
    rng = np.random.default_rng(16)
    q, k, v = (rounded(rng.normal(0, 1, (n, 2, dim)).astype(np.float32), t) for _ in range(3))
    bad = q.copy()
    good = np.ones((n, 2), bool)
    for r, h, e, x in ((0, 0, 5, np.nan), (1, 1, 0, np.nan), (n // 2, 0, dim - 1, np.nan), (n - 1, 1, 7, -np.nan)):
        bad[r, h, e] = x
        good[r, h] = False
    seen = np.tril(np.ones((n, n), bool)) if causal else None
    got, lse = prompt(*(cuda(x).to(dtype(t)) for x in (bad, k, v)), [0, n], [0, n], causal)
    check_rows(got, lse, q, k, v, seen, t, good)


@pytest.mark.parametrize("at", [0, 1, 5, 17, 40, 127, 130, 299])
@pytest.mark.parametrize("dim,t,causal", [(64, "f16", True), (128, "bf16", True), (128, "f16", False)])
def test_prompt_nan_in_a_key_makes_the_rows_that_see_it_nan(dim, t, causal, at):
    """In every kind of column: the exponential is computed in two ways."""
    n = 300
    rng = np.random.default_rng(17)
    q, k, v = (rounded(rng.normal(0, 1, (n, 2, dim)).astype(np.float32), t) for _ in range(3))
    bad = k.copy()
    bad[at, 1, 3] = np.nan
    good = np.ones((n, 2), bool)
    good[at if causal else 0:, 1] = False
    seen = np.tril(np.ones((n, n), bool)) if causal else None
    got, lse = prompt(*(cuda(x).to(dtype(t)) for x in (q, bad, v)), [0, n], [0, n], causal)
    check_rows(got, lse, q, k, v, seen, t, good)


@pytest.mark.parametrize("at", [2, 40, 200])
@pytest.mark.parametrize("dim,t", [(64, "bf16"), (128, "bf16"), (128, "f16")])
def test_prompt_infinite_scores(dim, t, at):
    """One infinite element of a key: a score of +infinity has no softmax (NaN), one of -infinity is a key without weight."""
    n = 300
    rng = np.random.default_rng(18)
    q, k, v = (rounded(rng.normal(0, 1, (n, 2, dim)).astype(np.float32), t) for _ in range(3))
    bad = k.copy()
    bad[at, 0, 9] = np.inf
    seen = np.tril(np.ones((n, n), bool))
    good = ~(seen[:, at][:, None] & (q[:, :, 9] > 0) & (np.arange(2) == 0))
    assert np.all(q[:, 0, 9] != 0) and (~good).any() and good[at:, 0].any()
    got, lse = prompt(*(cuda(x).to(dtype(t)) for x in (q, bad, v)), [0, n], [0, n])
    for h, s in ((0, seen & (np.arange(n) != at)), (1, seen)):
        low = good[:, h].copy()
        if h == 0:
            low[:at] = True
        check_rows(got[:, h:h + 1], lse[:, h:h + 1], q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], s, t, low[:, None])


@pytest.mark.parametrize("dim,t,lq,lk,group", [
    (64, "f16", 300, 300, 2), (64, "bf16", 250, 300, 3), (128, "bf16", 300, 300, 2), (128, "f16", 100, 333, 4),
    (128, "bf16", 400, 400, 1), (64, "f16", 400, 130, 1), (128, "bf16", 5, 5, 4),
])
def test_values_that_a_row_does_not_see_may_be_anything(dim, t, lq, lk, group):
    """NaN and infinities among the values: a row before them keeps its bits; one that sees them has NaN, or the
    infinity, in their columns, and keeps the bits of the others."""
    tt = torch()
    rng = np.random.default_rng(19)
    hk = 2
    q = cuda(rng.normal(0, 1, (lq, hk * group, dim)).astype(np.float32)).to(dtype(t))
    k, v = (cuda(rng.normal(0, 1, (lk, hk, dim)).astype(np.float32)).to(dtype(t)) for _ in range(2))
    clean, lse = prompt(q, k, v, [0, lq], [0, lk])
    inf, nan = float("inf"), float("nan")
    marks = [(lk - 1, 0, 0, nan), (lk - 1, 1, dim - 1, inf), (max(0, lk - 2), 0, 1, -inf), (lk // 2, 0, 2, inf),
             (lk // 2 + 1, 0, 2, -inf), (lk * 2 // 3, 1, 33, nan), (lk * 3 // 4, 1, 8, -inf)]
    for many in (marks[:1], marks[1:2], marks):
        dirty = v.clone()
        first = np.full((hk, dim), lk + 1)
        for at, h, e, x in many:
            dirty[at, h, e] = x
            first[h, e] = min(first[h, e], at)
        got, l2 = prompt(q, k, dirty, [0, lq], [0, lk])
        assert tt.equal(l2, lse)
        last = np.arange(lq) + lk - lq  # the last key that a row sees
        sees = cuda(np.repeat(first, group, 0)[None] <= last[:, None, None])
        assert tt.equal(got[~sees], clean[~sees])
        assert not bool(tt.isfinite(got[sees]).any())
    # the whole of the last row, seen by the last query alone (or by none)
    dirty = v.clone()
    dirty[lk - 1] = nan
    got, _ = prompt(q, k, dirty, [0, lq], [0, lk])
    assert tt.equal(got[:lq - 1], clean[:lq - 1]) and bool(tt.isnan(got[lq - 1]).all())


@pytest.mark.parametrize("dim,t", [(64, "f16"), (128, "bf16")])
def test_an_infinite_value_is_the_rows_that_see_it(dim, t):
    """Around the diagonal the sign is kept: +inf, -inf, and NaN where both are seen."""
    n = 96
    rng = np.random.default_rng(20)
    q, k, v = (cuda(rng.normal(0, 1, (n, 1, dim)).astype(np.float32)).to(dtype(t)) for _ in range(3))
    v[50, 0, 3], v[60, 0, 3], v[70, 0, 4] = float("inf"), float("-inf"), float("-inf")
    got, _ = prompt(q, k, v, [0, n], [0, n])
    g = to_np(got)[:, 0]
    assert np.isfinite(g[:50]).all() and np.isposinf(g[50:60, 3]).all() and np.isnan(g[60:, 3]).all()
    assert np.isfinite(g[:70, 4]).all() and np.isneginf(g[70:, 4]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [12.0, 18.0, 22.0, 25.0])
def test_prompt_fp16_weights_far_below_the_largest(dim, gap):
    """One key with nearly all the weight and a value of 0, 4095 others 2^-gap below it that make up the output.

    A weight is held in fp16 at 2^7 times its size relative to the row's reference (which the largest weight exceeds by
    2^8 at most, so that it stays below 2^15): within fp16's half step, 2^-11 of it, from 2^-21 of the largest up, and
    within half of fp16's smallest step below, 2^-25 / 2^7 = 2^-32 of the reference.  Here the first tile holds the
    largest score, which is the reference, so the floor is at most 2^-32 sum |v| (the sum of weights being at least 1)."""
    tt = torch()
    n, rows = 4096, 40
    rng = np.random.default_rng(21)
    q, k = np.zeros((rows, 1, dim), np.float32), np.zeros((n, 1, dim), np.float32)
    q[:, 0, 0], k[:, 0, 0] = 1.0, -gap / np.log2(np.e)
    q[:, 0, 1], k[:, 0, 1] = rng.uniform(0.5, 1, rows), rng.uniform(-1, 0, n)
    k[7] = 0.0
    v = rng.uniform(0.5, 1.5, (n, 1, dim)).astype(np.float32)
    v[7] = 0.0
    q, k, v = (rounded(x, "f16") for x in (q, k, v))
    got, _ = prompt(*(cuda(x).half() for x in (q, k, v)), [0, rows], [0, n], causal=False, scale=1.0)
    o, _, mag, size, _ = ref.attend(q, k, v, 1.0)
    floor = 2.0 ** -32 * np.abs(v.astype(np.float64)).sum(0)
    err = np.abs(to_np(got.double()) - o)
    tol = bound(mag, size, o, n, dim, half_step("f16"), "f32", floor)
    assert np.all(err <= tol), f"{np.max(err / tol):.3g} of the bound"


@pytest.mark.parametrize("dim,t,group", [(128, "f32", 4), (128, "bf16", 1), (64, "f16", 8), (64, "f32", 12)])
@pytest.mark.parametrize("bad", [np.nan, -np.nan, np.inf, -np.inf])
def test_decode_queries_that_are_not_finite(dim, t, group, bad):
    """The head's output and lse are NaN (an infinite query has scores of both signs here); the others keep their bits."""
    lens = [700, 1, 0, 5000, 33]
    cache, table, q = decode_case(dim, t, 16, 2, group, lens, seed=41)
    dev = dev_cache(cache)
    want, wl = run_decode(dev, q, lens, table, t)
    dirty = q.copy()
    good = np.ones(q.shape[:2], bool)
    for i, h, e in ((0, 0, 0), (3, group, dim - 1), (4, 2 * group - 1, 17), (2, 0, 3)):
        dirty[i, h, e] = bad
        good[i, h] = lens[i] == 0   # no keys: 0, whatever the query
    got, lse = run_decode(dev, dirty, lens, table, t)
    assert np.array_equal(got[good], want[good]) and np.array_equal(lse[good], wl[good])
    assert np.isnan(got[~good]).all() and np.isnan(lse[~good]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 3], [9, 1, 100]])
def test_append_of_numbers_that_are_not_finite(bad, side, new):
    """The block's scale is NaN, so that all that is read of it is; other heads and blocks keep the definition's bits, a
    later token of the block does not bring the scale back, and a page's next owner does."""
    b, tt = lib(), torch()
    dim, hk, group, page, old = 64, 3, 2, 32, [5, 0, 20]
    cache, table, qkv, _, _ = append_case(dim, "f32", 0, False, page, hk, group, [n + 1 for n in new], old, seed=51)
    n = sum(new)
    dev = dev_cache(cache)
    parts = [x[:n].copy() for x in split(qkv, hk * group, hk, dim)]
    dirty = [x.copy() for x in parts]
    which = 1 if side == "k" else 2
    cu = cu_of(new)
    at, head = int(cu[2]), 1      # the first new token of the last sequence: position 20, block 1, four older tokens
    dirty[which][at, head, 11] = bad
    outs = [tt.empty(x.shape, device="cuda") for x in parts]
    b.bitnet_kv_append(dev, *(cuda(x) for x in dirty), cuda(cu), ints(*old), cuda(table), *outs)
    ref.append(cache, *parts, cu, old, table)
    for o, x in zip(outs, dirty):
        same_bits(to_np(o), x, "outputs")

    def check(what):
        page0 = table[2][0]
        for name in ("k", "v", "k_scale", "v_scale"):
            got, want = to_np(getattr(dev, name)).copy(), getattr(cache, name).copy()
            if name[0] == side:
                if name[1:]:
                    assert np.isnan(got[page0, head, 1]), what
                    got[page0, head, 1] = want[page0, head, 1] = 0
                else:
                    got[page0, head, 16:32] = want[page0, head, 16:32] = 0
            same_bits(got, want, f"{what}: {name}")

    check("append")
    total = [a + c for a, c in zip(old, new)]
    rows = {s: tt.empty((sum(total), hk, dim), device="cuda") for s in "kv"}
    b.bitnet_kv_gather(dev, cuda(cu_of(total)), cuda(table), rows["k"], rows["v"])
    block = slice(sum(total[:2]) + 16, sum(total[:2]) + min(32, total[2]))
    for s in "kv":
        nan = tt.isnan(rows[s])
        want = tt.zeros_like(nan)
        if s == side:
            want[block, head] = True
        assert tt.equal(nan, want), s
    q = rounded(np.random.default_rng(3).normal(0, 1, (3, hk * group, dim)).astype(np.float32), "f32")
    got, lse = run_decode(dev, q, total, table, "f32")
    hurt = np.zeros(got.shape[:2], bool)
    hurt[2, head * group:(head + 1) * group] = True
    assert np.isnan(got[hurt]).all() and np.isfinite(got[~hurt]).all()
    assert np.isnan(lse[hurt]).all() if side == "k" else np.isfinite(lse).all()
    # one finite token more for each sequence
    more = [x[n:n + 3].copy() for x in split(qkv, hk * group, hk, dim)]
    b.bitnet_kv_append(dev, *(cuda(x) for x in more), ints(0, 1, 2, 3), ints(*total), cuda(table),
                       tt.empty((3, hk * group, dim), device="cuda"))
    ref.append(cache, *more, [0, 1, 2, 3], total, table)
    check("a token more")
    # the page from its start, by another sequence
    b.bitnet_kv_append(dev, *(cuda(x[:3]) for x in more), ints(0, 3), ints(16), cuda(table[2:]),
                       tt.empty((3, hk * group, dim), device="cuda"))
    ref.append(cache, *more, [0, 3], [16], table[2:])
    page0 = table[2][0]
    for name in ("k_scale", "v_scale"):
        assert np.isfinite(to_np(getattr(dev, name))[page0, :, 1]).all()
        same_bits(to_np(getattr(dev, name))[page0, :, 1], getattr(cache, name)[page0, :, 1], name)
    for name in ("k", "v"):
        same_bits(to_np(getattr(dev, name))[page0, :, 16:19], getattr(cache, name)[page0, :, 16:19], name)


@pytest.mark.parametrize("dim,t,lens", [(128, "f32", [5000, 900, 0]), (64, "bf16", [1]), (128, "f16", [40000])])
def test_decode_wait_that_runs_out(dim, t, lens):
    """A cap of one leaves no try: every warp with a tile gives up, waits for its copies and returns, and TIMEOUT is
    latched; the next call on the same workspace has the bits of one before."""
    b, tt = lib(), torch()
    cache, table, q = decode_case(dim, t, 32, 2, 4, lens, seed=61)
    dev = dev_cache(cache)
    ws = tt.zeros(b.bitnet_attn_decode_workspace_bytes(len(lens), 8, 2, dim), dtype=tt.uint8, device="cuda")
    want, wl = run_decode(dev, q, lens, table, t, ws)
    check_decode(cache, table, q, lens, t, want, wl)
    for _ in range(2):
        b.bitnet_set_wait_limit(1)
        try:
            for _ in range(4):
                run_decode(dev, q, lens, table, t, ws)
            st = b.bitnet_get_device_error()
        finally:
            b.bitnet_set_wait_limit(0)
        assert st == b.BITNET_ERR_TIMEOUT
        assert b.bitnet_get_device_error() == b.BITNET_OK
        got, lse = run_decode(dev, q, lens, table, t, ws)
        assert b.bitnet_get_device_error() == b.BITNET_OK
        assert np.array_equal(got, want) and np.array_equal(lse, wl)
    check_cache(dev, cache, "after")


@pytest.mark.parametrize("dim,t,hk,group,lens", [
    (128, "f32", 1, 4, [20] * 296 + [30000, 3, 15000, 0, 9000]),   # long ones beside each other and alone
    (128, "bf16", 2, 8, [17] * 100 + [20000] + [40] * 60),
    (64, "f16", 1, 12, [25000] + [30] * 300),                      # two chunks of heads, the first unit long
    (64, "f32", 4, 1, [0, 1] * 60 + [12000]),
])
def test_decode_a_long_sequence_among_many_short_ones(dim, t, hk, group, lens):
    """A unit in hundreds of parts among hundreds that lie in one: right, and the same bits again."""
    cache, table, q = decode_case(dim, t, 64, hk, group, lens, seed=71)
    dev = dev_cache(cache)
    got, lse = run_decode(dev, q, lens, table, t)
    check_decode(cache, table, q, lens, t, got, lse)
    again, l2 = run_decode(dev, q, lens, table, t)
    assert np.array_equal(got, again) and np.array_equal(lse, l2)


def test_captured_prompt_calls_serve_any_bounds():
    """Append, gather and prompt attention in one graph whose bounds and lengths are changed on the device between the
    replays: the bits of the same calls made directly, rows behind the last sequence left as they were."""
    b, tt = lib(), torch()
    rng = np.random.default_rng(81)
    dim, hk, group, page, seqs, rows = 128, 2, 2, 32, 3, 400
    hq = hk * group
    table = cuda(np.arange(seqs * 16, dtype=np.int32).reshape(seqs, 16))
    qkv = cuda(rng.normal(0, 1, (rows, (hq + 2 * hk) * dim)).astype(np.float32))
    rope = cuda(ref.angles(600, dim))
    cu, old, cu_k = ints(0, 0, 0, 0), ints(0, 0, 0), ints(0, 0, 0, 0)

    def state():
        dev = dev_cache(ref.Cache(seqs * 16, hk, page, dim))
        return dev, tt.zeros((rows, hq, dim), device="cuda").half(), \
            [tt.zeros((2 * rows, hk, dim), device="cuda").half() for _ in range(2)], tt.zeros((rows, hq, dim), device="cuda")

    def calls(dev, q16, kv, out):
        b.bitnet_kv_append(dev, *split(qkv, hq, hk, dim), cu, old, table, q16, rope=rope)
        b.bitnet_kv_gather(dev, cu_k, table, *kv)
        b.bitnet_attn_prompt(q16, *kv, cu, cu_k, out)

    direct, captured = state(), state()
    side, graph = tt.cuda.Stream(), tt.cuda.CUDAGraph()
    side.wait_stream(tt.cuda.current_stream())
    with tt.cuda.graph(graph, stream=side):
        calls(*captured)
    tt.cuda.current_stream().wait_stream(side)
    lengths = np.zeros(seqs, np.int32)
    for new in ([100, 1, 150], [0, 250, 17], [1, 1, 1], [130, 0, 0]):
        cu.copy_(cuda(cu_of(new)))
        old.copy_(cuda(lengths))
        lengths = lengths + np.array(new, np.int32)
        cu_k.copy_(cuda(cu_of(lengths)))
        for st in (direct, captured):
            st[3].fill_(9.0)
        calls(*direct)
        graph.replay()
        tt.cuda.synchronize()
        assert b.bitnet_get_device_error() == b.BITNET_OK
        for n in ("k", "v", "k_scale", "v_scale"):
            assert tt.equal(getattr(direct[0], n), getattr(captured[0], n)), n
        for x, y in zip((direct[1], *direct[2], direct[3]), (captured[1], *captured[2], captured[3])):
            assert tt.equal(x, y)
        assert bool((captured[3][sum(new):] == 9).all()) and bool(tt.isfinite(captured[3]).all())


def test_prompt_calls_side_by_side():
    """Both head sizes and the three packed calls on two streams at once: the bits of the calls alone."""
    b, tt = lib(), torch()
    g = tt.Generator(device="cuda")
    g.manual_seed(91)
    calls, outs, want = [], [], []
    for dim, dt, lens in ((64, tt.float16, [700, 1, 333]), (128, tt.bfloat16, [40, 900])):
        n = sum(lens)
        q = tt.randn((n, 4, dim), generator=g, device="cuda").to(dt)
        k, v = (tt.randn((n, 2, dim), generator=g, device="cuda").to(dt) for _ in range(2))
        cu, table = cuda(cu_of(lens)), tt.arange(len(lens) * 32, dtype=tt.int32, device="cuda").view(len(lens), 32)
        dev, zero = dev_cache(ref.Cache(len(lens) * 32, 2, 32, dim)), ints(*[0] * len(lens))
        out, rows, k16 = tt.empty_like(q), [tt.empty_like(k) for _ in range(2)], tt.empty_like(k)

        def call(stream, q=q, k=k, v=v, cu=cu, table=table, dev=dev, zero=zero, out=out, rows=rows, k16=k16):
            b.bitnet_kv_append(dev, None, k, v, cu, zero, table, None, k_out=k16, stream=stream)
            b.bitnet_kv_gather(dev, cu, table, *rows, stream=stream)
            b.bitnet_attn_prompt(q, *rows, cu, cu, out, stream=stream)

        calls.append(call)
        outs.append((out, *rows, dev.k, dev.v_scale))
        call(None)
        tt.cuda.synchronize()
        want.append([x.clone() for x in outs[-1]])
    streams = [tt.cuda.Stream() for _ in range(2)]
    for x in outs:
        x[0].zero_()
    tt.cuda.synchronize()
    for _ in range(20):
        for call, stream in zip(calls, streams):
            call(stream)
    tt.cuda.synchronize()
    assert b.bitnet_get_device_error() == b.BITNET_OK
    for got, ref_ in zip(outs, want):
        for x, y in zip(got, ref_):
            assert tt.equal(x, y)
