"""Host-side checks of the cache and attention calls: every refusal happens before
the GPU is touched (fake device addresses, no GPU needed), the binding's structs
have the header's layout, and the plain implementation that the GPU tests use
does what the definitions say."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import attn_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a fake device address, never dereferenced on the host


@pytest.fixture(scope="module")
def b():
    import ternary_weight_absmax_b200 as mod
    return mod


def cache(b, **kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, num_pages=4, kv_heads=2, head_dim=128, page_size=16)
    f.update(kw)
    return b.bitnet_kv_cache(**f)


def append_args(b, **kw):
    f = dict(q=A, k=A, v=A, q_stride=1024, k_stride=1024, v_stride=1024, tokens=3, cu_tokens=A, cache_len=A, block_table=A,
             rope=A, rope_rows=100, rot_dim=128, q_out=A, q_heads=4, seqs=2, max_pages=3, eps=1e-6,
             in_dtype=b.BITNET_F32, out_dtype=b.BITNET_F32)
    f.update(kw)
    return b.bitnet_kv_append_args(**f)


def prompt_args(b, **kw):
    f = dict(q=A, k=A, v=A, q_stride=1024, k_stride=1024, v_stride=1024, q_tokens=3, k_tokens=3, cu_q=A, cu_k=A, out=A,
             scale=0.1, seqs=1, q_heads=4, kv_heads=2, head_dim=128, causal=1, dtype=b.BITNET_BF16,
             out_dtype=b.BITNET_BF16)
    f.update(kw)
    return b.bitnet_attn_prompt_args(**f)


BAD_CACHES = [("BITNET_ERR_NULL", dict(k=None)), ("BITNET_ERR_NULL", dict(v_scale=None)),
              ("BITNET_ERR_SHAPE", dict(head_dim=96)), ("BITNET_ERR_SHAPE", dict(kv_heads=0)),
              ("BITNET_ERR_SHAPE", dict(page_size=8)), ("BITNET_ERR_SHAPE", dict(page_size=48)),
              ("BITNET_ERR_SHAPE", dict(page_size=2048)), ("BITNET_ERR_SHAPE", dict(num_pages=0)),
              ("BITNET_ERR_SHAPE", dict(num_pages=1 << 26)),
              ("BITNET_ERR_ALIGN", dict(k=A + 8)), ("BITNET_ERR_ALIGN", dict(k_scale=A + 2))]


@pytest.mark.parametrize("status,kw", BAD_CACHES)
def test_bad_caches(b, status, kw):
    lib, c = b.library(), ctypes.byref(cache(b, **kw))
    want = getattr(b, status)
    assert lib.bitnet_kv_append(c, ctypes.byref(append_args(b)), None) == want
    assert lib.bitnet_kv_gather(c, A, A, 1, 1, 4, A, A, 0, None) == want
    assert lib.bitnet_attn_decode(c, A, 512, 4, A, A, 1, 1, 0.1, A, None, 0, A, 1 << 30, None) == want
    assert b.bitnet_last_error_detail()


@pytest.mark.parametrize("status,kw", [
    ("BITNET_ERR_SHAPE", dict(tokens=-1)), ("BITNET_ERR_SHAPE", dict(seqs=0)), ("BITNET_ERR_SHAPE", dict(max_pages=0)),
    ("BITNET_ERR_VALUE", dict(in_dtype=3)), ("BITNET_ERR_VALUE", dict(out_dtype=-1)),
    ("BITNET_ERR_NULL", dict(q_out=None)), ("BITNET_ERR_NULL", dict(q=None)), ("BITNET_ERR_NULL", dict(q_heads=0)),
    ("BITNET_ERR_SHAPE", dict(q_heads=3)), ("BITNET_ERR_SHAPE", dict(rot_dim=12)), ("BITNET_ERR_SHAPE", dict(rot_dim=136)),
    ("BITNET_ERR_SHAPE", dict(rot_dim=0)), ("BITNET_ERR_SHAPE", dict(rope=None)), ("BITNET_ERR_SHAPE", dict(rope_rows=0)),
    ("BITNET_ERR_NULL", dict(k=None)), ("BITNET_ERR_ALIGN", dict(v=A + 8)), ("BITNET_ERR_ALIGN", dict(k_stride=1022)),
    ("BITNET_ERR_SHAPE", dict(q_stride=508)), ("BITNET_ERR_NULL", dict(cu_tokens=None)),
    ("BITNET_ERR_NULL", dict(block_table=None)), ("BITNET_ERR_ALIGN", dict(cache_len=A + 1)),
    ("BITNET_ERR_ALIGN", dict(k_out=A + 8)), ("BITNET_ERR_ALIGN", dict(q_norm=A + 4)), ("BITNET_ERR_ALIGN", dict(rope=A + 4)),
])
def test_bad_appends(b, status, kw):
    got = b.library().bitnet_kv_append(ctypes.byref(cache(b)), ctypes.byref(append_args(b, **kw)), None)
    assert got == getattr(b, status), b.bitnet_last_error_detail()


@pytest.mark.parametrize("eps", [-1e-6, float("nan"), float("inf")])
def test_append_refuses_an_eps_that_no_norm_has(b, eps):
    lib, c = b.library(), ctypes.byref(cache(b))
    for norm in ("q_norm", "k_norm"):
        a = append_args(b, eps=eps, tokens=0, **{norm: A})
        assert lib.bitnet_kv_append(c, ctypes.byref(a), None) == b.BITNET_ERR_VALUE
    assert lib.bitnet_kv_append(c, ctypes.byref(append_args(b, eps=eps, tokens=0)), None) == b.BITNET_OK


def test_null_and_empty(b):
    lib, c = b.library(), ctypes.byref(cache(b))
    assert lib.bitnet_kv_append(None, ctypes.byref(append_args(b)), None) == b.BITNET_ERR_NULL
    assert lib.bitnet_kv_append(c, None, None) == b.BITNET_ERR_NULL
    assert lib.bitnet_attn_prompt(None, None) == b.BITNET_ERR_NULL
    assert lib.bitnet_kv_append(c, ctypes.byref(append_args(b, tokens=0)), None) == b.BITNET_OK
    assert lib.bitnet_kv_gather(c, None, None, 1, 1, 0, None, None, 0, None) == b.BITNET_OK
    assert lib.bitnet_attn_prompt(ctypes.byref(prompt_args(b, q_tokens=0)), None) == b.BITNET_OK


def test_bad_gathers_and_decodes(b):
    lib, c = b.library(), ctypes.byref(cache(b))
    assert lib.bitnet_kv_gather(c, A, A, 0, 1, 4, A, A, 0, None) == b.BITNET_ERR_SHAPE
    assert lib.bitnet_kv_gather(c, A, A, 1, 1, -4, A, A, 0, None) == b.BITNET_ERR_SHAPE
    assert lib.bitnet_kv_gather(c, A, A, 1, 1, 4, A, A, 5, None) == b.BITNET_ERR_VALUE
    assert lib.bitnet_kv_gather(c, A, A, 1, 1, 4, None, A, 0, None) == b.BITNET_ERR_NULL
    assert lib.bitnet_kv_gather(c, A, A, 1, 1, 4, A, A + 8, 0, None) == b.BITNET_ERR_ALIGN
    need = b.bitnet_attn_decode_workspace_bytes(1, 4, 2, 128)
    assert need > 0 and b.bitnet_attn_decode_workspace_bytes(9999, 4, 2, 128) >= need
    assert b.bitnet_attn_decode_workspace_bytes(1, 5, 2, 128) == 0
    assert b.bitnet_attn_decode_workspace_bytes(1, 4, 2, 96) == 0

    def decode(q=A, stride=512, heads=4, lens=A, table=A, seqs=1, pages=1, scale=0.1, out=A, lse=None, dt=0, ws=A, n=need):
        return lib.bitnet_attn_decode(c, q, stride, heads, lens, table, seqs, pages, scale, out, lse, dt, ws, n, None)

    assert decode(heads=3) == b.BITNET_ERR_SHAPE
    assert decode(seqs=0) == b.BITNET_ERR_SHAPE
    assert decode(pages=0) == b.BITNET_ERR_SHAPE
    assert decode(dt=7) == b.BITNET_ERR_VALUE
    assert decode(scale=float("nan")) == b.BITNET_ERR_VALUE
    assert decode(scale=float("inf")) == b.BITNET_ERR_VALUE
    assert decode(q=None) == b.BITNET_ERR_NULL
    assert decode(q=A + 8) == b.BITNET_ERR_ALIGN
    assert decode(q=A + 4, dt=1) == b.BITNET_ERR_ALIGN
    assert decode(stride=508, seqs=2) == b.BITNET_ERR_SHAPE
    assert decode(stride=514) == b.BITNET_ERR_ALIGN
    assert decode(out=None) == b.BITNET_ERR_NULL
    assert decode(out=A + 4) == b.BITNET_ERR_ALIGN
    assert decode(lse=A + 2) == b.BITNET_ERR_ALIGN
    assert decode(ws=None) == b.BITNET_ERR_NULL
    assert decode(ws=A + 8) == b.BITNET_ERR_ALIGN
    assert decode(n=need - 1) == b.BITNET_ERR_BUFSIZE


@pytest.mark.parametrize("status,kw", [
    ("BITNET_ERR_SHAPE", dict(head_dim=80)), ("BITNET_ERR_SHAPE", dict(kv_heads=0)), ("BITNET_ERR_SHAPE", dict(q_heads=5)),
    ("BITNET_ERR_SHAPE", dict(seqs=0)), ("BITNET_ERR_SHAPE", dict(q_tokens=-1)), ("BITNET_ERR_SHAPE", dict(k_tokens=-1)),
    ("BITNET_ERR_VALUE", dict(dtype=0)), ("BITNET_ERR_VALUE", dict(out_dtype=2)), ("BITNET_ERR_VALUE", dict(scale=float("inf"))),
    ("BITNET_ERR_NULL", dict(q=None)), ("BITNET_ERR_NULL", dict(v=None)), ("BITNET_ERR_ALIGN", dict(k=A + 8)),
    ("BITNET_ERR_ALIGN", dict(q_stride=1020)), ("BITNET_ERR_SHAPE", dict(k_stride=248)), ("BITNET_ERR_NULL", dict(cu_k=None)),
    ("BITNET_ERR_NULL", dict(out=None)), ("BITNET_ERR_ALIGN", dict(out=A + 8)), ("BITNET_ERR_ALIGN", dict(lse=A + 2)),
    ("BITNET_ERR_SHAPE", dict(q_tokens=1 << 30, q_heads=1024, kv_heads=1, q_stride=1 << 20)),
])
def test_bad_prompts(b, status, kw):
    got = b.library().bitnet_attn_prompt(ctypes.byref(prompt_args(b, **kw)), None)
    assert got == getattr(b, status), b.bitnet_last_error_detail()


def test_struct_layouts_match_the_header(b, tmp_path):
    fields = {n: [f for f, _ in getattr(b, n)._fields_]
              for n in ("bitnet_kv_cache", "bitnet_kv_append_args", "bitnet_attn_prompt_args")}
    src = tmp_path / "layout.c"
    body = "".join(f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for s, fs in fields.items() for f in fs)
    body += "".join(f'printf("{s} %zu\\n", sizeof({s}));' for s in fields)
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bitnet_w2a8.h"\nint main(void) {' + body + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, n = line.split()
        s, _, f = name.partition(".")
        t = getattr(b, s)
        assert int(n) == (getattr(t, f).offset if f else ctypes.sizeof(t)), name


def test_binding_refuses_what_the_call_cannot_see(b):
    import torch
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        b.KVCache(torch.zeros(1, 1, 16, 64, dtype=torch.int8), torch.zeros(1, 1, 16, 64, dtype=torch.int8),
                  torch.ones(1, 1, 1), torch.ones(1, 1, 1))
    with pytest.raises(ValueError, match="pages"):
        b.KVCache(torch.zeros(4), torch.zeros(4), torch.ones(1), torch.ones(1))
    with pytest.raises(ValueError, match="CUDA"):
        b.bitnet_attn_prompt(x.half(), x.half(), x.half(), torch.zeros(2, dtype=torch.int32),
                             torch.zeros(2, dtype=torch.int32), x.half())


def test_reference_append_keeps_values_within_half_a_code():
    rng = np.random.default_rng(1)
    c = ref.Cache(6, 2, 16, 64)
    table = ref.tables(rng, [3, 3], 6)
    k, v = (rng.normal(0, 1, (70, 2, 64)).astype(np.float32) for _ in range(2))
    ref.append(c, None, k, v, [0, 40, 70], [0, 0], table)
    for i, (a, n) in enumerate(((0, 40), (40, 30))):
        for side, x in (("k", k), ("v", v)):
            got = c.rows(side, table[i], n)
            for t in range(0, n, 16):
                w = x[a + t:a + min(n, t + 16)]
                step = np.abs(w).max((0, 2)) / 127
                assert np.all(np.abs(got[t:t + 16][:w.shape[0]] - w) <= 0.5001 * step[None, :, None])


def test_reference_append_in_two_calls_keeps_values_within_a_code():
    """A block filled by two calls has the scale of the larger; old codes are rounded twice."""
    rng = np.random.default_rng(2)
    c = ref.Cache(1, 1, 16, 64)
    k = rng.normal(0, 1, (16, 1, 64)).astype(np.float32)
    k[9:] *= 5
    for a, e in ((0, 9), (9, 16)):
        ref.append(c, None, k[a:e], k[a:e], [0, e - a], [a], np.array([[0]]))
    step = np.abs(k).max() / 127
    assert np.float32(127) * (np.float32(1) / np.abs(k).max()) == c.k_scale[0, 0, 0]
    assert np.all(np.abs(c.rows("k", [0], 16) - k) <= 1.001 * step)


def test_reference_rotation_keeps_lengths_and_turns_by_differences():
    """Scores of rotated vectors depend on the difference of positions, in both layouts."""
    rng = np.random.default_rng(3)
    rope = ref.angles(50, 64)
    x, y = (rng.normal(0, 1, (1, 64)).astype(np.float32) for _ in range(2))
    for inter in (False, True):
        at = [float((ref.norm_rotate(x, None, 0, rope[p], inter).astype(np.float64) *
                     ref.norm_rotate(y, None, 0, rope[p + 7], inter)).sum()) for p in (0, 5, 40)]
        assert np.ptp(at) < 1e-4
        assert abs(np.linalg.norm(ref.norm_rotate(x, None, 0, rope[31], inter)) - np.linalg.norm(x)) < 1e-5


def test_reference_attention_against_a_direct_sum():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(0, 1, (3, 4, 8)), rng.normal(0, 1, (5, 2, 8)), rng.normal(0, 1, (5, 2, 8))
    seen = np.arange(5)[None] <= np.arange(3)[:, None] + 2
    seen[0] = False
    out, lse, _, _, _ = ref.attend(q, k, v, 0.3, seen)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0]))
    for r in (1, 2):
        for h in range(4):
            w = [np.exp(0.3 * q[r, h] @ k[j, h // 2]) if seen[r, j] else 0.0 for j in range(5)]
            np.testing.assert_allclose(out[r, h], sum(w[j] * v[j, h // 2] for j in range(5)) / sum(w), rtol=1e-12)
            np.testing.assert_allclose(lse[r, h], np.log(sum(w)), rtol=1e-12)


def test_prompt_exponential_polynomial_is_within_its_stated_error():
    """The coefficients in the source, evaluated with fp32 roundings as the kernel does: 2^-18.4 of the fit, and
    half a step (2^-24) for each of five operations on values up to about 1.5 times the result."""
    import re
    import numpy as np
    src = open(os.path.join(ROOT, "ternary_weight_absmax_b200", "csrc", "attn_prompt.cu")).read()
    body = src[src.index("uint64_t ex2_poly"):]
    body = body[:body.index("\n}\n")]
    c = [np.float32(x) for x in re.findall(r"pack2\((0\.\d+)f, \1f\)", body)]
    assert len(c) == 4
    y = np.linspace(-125.9, 8.0, 400001).astype(np.float32)
    n = np.rint(y)
    r = (y - n).astype(np.float32)
    p = c[0]
    for k in (*c[1:], np.float32(1.0)):
        p = (p.astype(np.float64) * r + k).astype(np.float32)
    got = np.ldexp(p.astype(np.float64), n.astype(int))
    err = np.abs(got / np.exp2(y.astype(np.float64)) - 1.0).max()
    assert err <= 2.0 ** -18.4 + 5 * 1.5 * 2.0 ** -24


def test_prompt_exponential_polynomial_ends_in_zero():
    """Below the normal numbers: no sign or exponent bit is touched (at most 2^-126), and exactly 0 from -127 down."""
    import re
    import numpy as np
    src = open(os.path.join(ROOT, "ternary_weight_absmax_b200", "csrc", "attn_prompt.cu")).read()
    body = src[src.index("uint64_t ex2_poly"):]
    body = body[:body.index("\n}\n")]
    c = [np.float32(x) for x in re.findall(r"pack2\((0\.\d+)f, \1f\)", body)]
    low = np.float32(re.search(r"fmaxf\(a, (-\d+\.\d+)f\)", body).group(1))
    y = np.concatenate([np.linspace(-200.0, -125.0, 100001), [-127.0, -126.5, -126.0, -np.inf]]).astype(np.float32)
    x = np.maximum(y, low)
    t = (x + np.float32(12582912.0)).astype(np.float32)
    n = (t - np.float32(12582912.0)).astype(np.float32)
    r = (x - n).astype(np.float32)
    p = np.full_like(r, c[0])
    for k in (*c[1:], np.float32(1.0)):
        p = (p.astype(np.float64) * r + k).astype(np.float32)
    bits = (t.view(np.uint32) << np.uint32(23)) + p.view(np.uint32)
    assert (bits[y <= -127] == 0).all()
    small = bits[(y > -127) & (y < -126)].view(np.float32)
    assert (small >= 0).all() and (small <= 2.0 ** -126).all()


def test_prompt_exponential_polynomial_up_to_the_largest_weight():
    """Weights reach 2^(lag + up): the polynomial keeps its bound there, and fp16 holds them."""
    import re
    src = open(os.path.join(ROOT, "ternary_weight_absmax_b200", "csrc", "attn_prompt.cu")).read()
    top = sum(float(re.search(p, src).group(1)) for p in (r"kLag = (\d+\.\d)f", r"__half>::value \? (\d+\.\d)f"))
    body = src[src.index("uint64_t ex2_poly"):]
    c = [np.float32(x) for x in re.findall(r"pack2\((0\.\d+)f, \1f\)", body[:body.index("\n}\n")])]
    y = np.linspace(8.0, top + 2.0 ** -10, 100001).astype(np.float32)
    n = np.rint(y)
    r, p = (y - n).astype(np.float32), c[0]
    for k in (*c[1:], np.float32(1.0)):
        p = (p.astype(np.float64) * r + k).astype(np.float32)
    got = np.ldexp(p.astype(np.float64), n.astype(int))
    assert np.abs(got / np.exp2(y.astype(np.float64)) - 1.0).max() <= 2.0 ** -18.4 + 5 * 1.5 * 2.0 ** -24
    assert got.max() < 65504


def test_traffic_records_belong_to_the_sources():
    """A capture counts only for the sources that it was made of: what other kernels need stays out of their headers,
    or the capture is made again."""
    import json
    import sys
    sys.path.insert(0, ROOT)
    import bench
    for kernel, d in json.load(open(os.path.join(ROOT, "profiles", "traffic.json"))).items():
        traffic, note = bench.read_traffic(kernel, d["algorithmic_bytes"])
        assert traffic == d["dram_bytes"], f"{kernel}: {note}"


def test_no_non_coherent_loads_beside_the_append():
    """The cache and attention kernels start while the kernel before them still writes (dependent launch); what they read
    after their wait may not go through the path for memory that is constant as long as a kernel runs."""
    import re
    csrc = os.path.join(ROOT, "ternary_weight_absmax_b200", "csrc")
    for n in ("attn.cuh", "attn_decode.cu", "attn_prompt.cu", "kv_cache.cu"):
        src = open(os.path.join(csrc, n)).read()
        assert not re.search(r"__ldg\b|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__", src), n


@pytest.mark.parametrize("dim,keys,stages", [(64, 64, 6), (128, 128, 4)])
def test_prompt_guarded_tiles_fit_their_barriers(dim, keys, stages):
    """The prompt kernel's count of tiles that a row sees in part, and how far two slots' walks are apart, over the
    shapes that can differ: the bounds that its barriers and a phase rely on."""
    import re
    src = open(os.path.join(ROOT, "ternary_weight_absmax_b200", "csrc", "attn_prompt.cu")).read()
    most_guarded = int(re.search(r"kGuarded = (\d+);", src).group(1))
    rng = np.random.default_rng(1)
    worst = 0
    for _ in range(60000):
        lq, lk, group = (int(x) for x in (rng.integers(1, 700), rng.integers(0, 900), rng.integers(1, 4)))
        causal = bool(rng.integers(0, 4))
        items = -(-lq // 128) * group
        pair = int(rng.integers(0, (items + 1) // 2))
        shift, row0, tiles = lk - lq, [], []
        for item in (2 * pair, 2 * pair + 1):
            r = item // group * 128
            seen = min(lk, min(r + 128, lq) + shift) if causal else lk
            tiles.append(-(-seen // keys) if item < items and seen > 0 else 0)
            row0.append(r)
        guard0 = max(0, min(lk, row0[0] + shift + 1) if causal else lk) // keys
        worst = max(worst, max(tiles) - guard0)
        for s in range(2):
            if tiles[s]:
                assert max(tiles) - tiles[s] < stages // 2
                last = min(lq, row0[s] + 128)
                for r in (row0[s], last - 1):   # before guard0 every row sees the whole tile
                    assert guard0 * keys <= max(0, min(lk, r + shift + 1) if causal else lk)
    assert worst <= most_guarded
