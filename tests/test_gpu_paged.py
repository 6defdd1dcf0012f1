"""Norm, rotation and the paged INT4 cache on the GPU against the oracle (float64).

k leaves the kernel as float64 arithmetic rounded to float32 and that to float16, so k,
codes and scales must match bit for bit. q is computed in float32: with h the exact
product x * w, its value h_a c - h_b s and the norm carry at most 8 roundings of 2^-24
relative to (|h_a| + |h_b|) r (sum of 4 partial butterfly terms, square root, division,
two products, an addition, the final product), then one float16 rounding of half a
step 2^-11 (subnormal results: 2^-25).
"""

import numpy as np
import pytest

import oracle
from gpu_util import say, to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import w4a16_decode_amd as q4mod

    say("libq4", q4mod.version())
    return q4mod


def _qkv(tokens, hq, hkv, d, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((tokens, hq + 2 * hkv, d)) * np.exp(r.standard_normal((1, hq + 2 * hkv, d)))
    return x.astype(np.float16)


def _table(rows, rot):
    a = oracle.paged.rope_angles(np.arange(rows), rot)
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def _same_bits(a, b):
    return np.array_equal(np.asarray(a).view(np.uint16), np.asarray(b).view(np.uint16))


def _check_q(got, x, weight, eps, cos, sin, interleaved, ref):
    mag = np.abs(oracle.paged.norm_rope(np.abs(x.astype(np.float64)), None if weight is None else np.abs(weight), eps))
    pair = np.broadcast_to(np.max(mag, axis=-1, keepdims=True), ref.shape)     # >= either of a pair
    err = np.abs(got.astype(np.float64) - ref)
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 8 * 2.0 ** -24 * 2 * pair
    assert np.all(err <= bound), (err / bound).max()


CASES = [  # tokens, hq, hkv, d, rot, interleaved, norm
    (1, 32, 8, 128, 128, False, True),
    (1, 1, 1, 64, 16, True, True),
    (7, 7, 1, 64, 64, False, True),
    (33, 6, 3, 128, 64, True, True),
    (5, 3, 3, 256, 256, False, True),
    (130, 8, 2, 256, 96, True, False),
    (17, 5, 1, 128, 32, False, False),
    (3, 9, 3, 64, 0, False, True),
    (2000, 4, 1, 128, 128, False, True),
]


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,interleaved,norm", CASES)
def test_qk_norm_rope(q4, tokens, hq, hkv, d, rot, interleaved, norm):
    import torch

    say("qk_norm_rope", tokens, hq, hkv, d, rot, interleaved, norm)
    x = _qkv(tokens, hq, hkv, d, seed=tokens + d)
    r = np.random.default_rng(1)
    wq, wk = ((1 + 0.3 * r.standard_normal(d)).astype(np.float16) if norm else None for _ in range(2))
    pos = r.integers(0, 4000, tokens).astype(np.int32)
    table = _table(4000, rot) if rot else None
    cos, sin = (table[pos, :, 0], table[pos, :, 1]) if rot else (None, None)
    g = to_gpu(x)
    before = g.clone()
    q, k = q4.qk_norm_rope(g[:, :hq], g[:, hq:hq + hkv], to_gpu(pos) if rot else None, to_gpu(table) if rot else None,
                           to_gpu(wq) if norm else None, to_gpu(wk) if norm else None, 1e-5, interleaved)
    ref_q = oracle.paged.norm_rope(x[:, :hq], wq, 1e-5, cos, sin, interleaved)
    ref_k = oracle.paged.norm_rope(x[:, hq:hq + hkv], wk, 1e-5, cos, sin, interleaved)
    assert _same_bits(to_np(k), ref_k.astype(np.float32).astype(np.float16))
    _check_q(to_np(q), x[:, :hq], wq, 1e-5, cos, sin, interleaved, ref_q)
    assert torch.equal(g, before)
    # in place, on the fused rows: the same bits, v untouched
    q4.qk_norm_rope(g[:, :hq], g[:, hq:hq + hkv], to_gpu(pos) if rot else None, to_gpu(table) if rot else None,
                    to_gpu(wq) if norm else None, to_gpu(wk) if norm else None, 1e-5, interleaved, g[:, :hq],
                    g[:, hq:hq + hkv])
    assert torch.equal(g[:, :hq], q) and torch.equal(g[:, hq:hq + hkv], k)
    assert torch.equal(g[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.parametrize("theta,rot", [(10000.0, 128), (500000.0, 64), (1.0, 16)])
def test_rope_table(q4, theta, rot):
    """float32 rounding (2^-25 of values up to 1) plus the angle's float64 error (positions
    below 2^17: an angle below 2^17 to ~4 * 2^-53 relative, 2^-34 absolute)."""
    n = 131072
    got = to_np(q4.rope_table(n, rot, theta))
    rows = np.concatenate([np.arange(50), np.random.default_rng(0).integers(0, n, 200), [n - 1]])
    a = oracle.paged.rope_angles(rows, rot, theta)
    assert np.abs(got[rows, :, 0] - np.cos(a)).max() <= 2.0 ** -25 + 2.0 ** -33
    assert np.abs(got[rows, :, 1] - np.sin(a)).max() <= 2.0 ** -25 + 2.0 ** -33
    assert tuple(q4.rope_table(0, rot, theta).shape) == (0, rot // 2, 2)


def test_positions_outside_the_table(q4):
    """A position outside the table is taken as the nearest inside."""
    import torch

    x = to_gpu(_qkv(4, 2, 1, 64, 3))
    table = q4.rope_table(10, 64)
    a = q4.qk_norm_rope(x[:, :2], x[:, 2:3], to_gpu(np.array([-5, 10, 2 ** 31 - 1, -2 ** 31], np.int32)), table)
    b = q4.qk_norm_rope(x[:, :2], x[:, 2:3], to_gpu(np.array([0, 9, 9, 0], np.int32)), table)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _cache_bytes(cache, k16, v16, slots, fill):
    """The cache's expected contents after storing the rows at the slots."""
    pages, heads, page, d, g = cache.pages, cache.kv_heads, cache.page_size, cache.head_dim, cache.group
    tiles = page // 16
    out = []
    for x in (k16, v16):
        codes, scales, values = oracle.paged.store(x, g)
        q = np.full((pages * page, heads, d), fill % 16 - 8)
        q[slots] = codes
        by_tile = q.reshape(pages, tiles, 16, heads, d).transpose(0, 3, 1, 2, 4).reshape(-1, 16, d)
        b = np.stack([oracle.paged.tile_bytes(t, x is v16) for t in by_tile]).reshape(pages, heads, page * d // 2)
        s = np.full((pages * page, heads, d // g), np.float16(7.0))
        s[slots] = scales
        s = s.reshape(pages, tiles, 16, heads, d // g).transpose(0, 3, 1, 4, 2).reshape(pages, heads, -1)
        out += [b, s, values]
    return out


@pytest.mark.parametrize("d,g,page", [(64, 32, 16), (64, 64, 48), (128, 128, 32), (128, 32, 16), (128, 64, 64),
                                      (256, 128, 16), (256, 32, 32)])
def test_append_bytes(q4, d, g, page):
    """Codes and scales of a scattered append, byte by byte; slots not written and padded
    rows (-1 and past the end) leave the cache as it was; dequant returns the values."""
    say("append", d, g, page)
    heads, pages, n = 3, 5, 37
    cache = q4.paged_kv_alloc(pages, page, heads, d, g)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x33)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(7.0)
    r = np.random.default_rng(d + g)
    x = _qkv(n, 2, heads, d, seed=d * g)
    x[3] = 0                                               # an all-zero token: scale 0
    x[4] *= np.float16(2.0 ** -14)                         # subnormal scales
    x[5] = (r.integers(-15, 16, x[5].shape) * 0.5).astype(np.float16)          # ties
    slots = r.permutation(pages * page)[:n].astype(np.int32)
    slots[[2, 9, 20]] = [-1, pages * page, 2 ** 31 - 1]
    kept = np.array([i for i in range(n) if i not in (2, 9, 20)])
    g_x = to_gpu(x)
    q4.paged_kv_append(g_x[:, 2:2 + heads], g_x[:, 2 + heads:], cache, to_gpu(slots))
    kc, ks, kv, vc, vs, vv = _cache_bytes(cache, x[kept, 2:2 + heads], x[kept, 2 + heads:], slots[kept], 0x33)
    assert np.array_equal(to_np(cache.k_codes), kc) and np.array_equal(to_np(cache.v_codes), vc)
    assert _same_bits(to_np(cache.k_scales), ks) and _same_bits(to_np(cache.v_scales), vs)
    back_k, back_v = (to_np(t) for t in q4.paged_kv_dequant(cache, to_gpu(slots)))
    assert _same_bits(back_k[kept] + np.float16(0), kv.astype(np.float16) + np.float16(0))
    assert _same_bits(back_v[kept] + np.float16(0), vv.astype(np.float16) + np.float16(0))
    assert not back_k[[2, 9, 20]].any() and not back_v[[2, 9, 20]].any()


@pytest.mark.parametrize("tokens,hq,hkv,d,rot,interleaved,norm", CASES)
def test_fused_append_is_the_two_steps(q4, tokens, hq, hkv, d, rot, interleaved, norm):
    """qk_norm_rope_append = qk_norm_rope, then paged_kv_append: the same bits."""
    import torch

    x = to_gpu(_qkv(tokens, hq, hkv, d, seed=7 * tokens + d))
    r = np.random.default_rng(2)
    w = [to_gpu((1 + 0.3 * r.standard_normal(d)).astype(np.float16)) if norm else None for _ in range(2)]
    pos = to_gpu(r.integers(0, 500, tokens).astype(np.int32)) if rot else None
    table = to_gpu(_table(500, rot)) if rot else None
    pages = -(-tokens // 16) + 1
    caches = [q4.paged_kv_alloc(pages, 16, hkv, d, 32) for _ in range(2)]
    slots = r.permutation(pages * 16)[:tokens].astype(np.int32)
    if tokens > 2:
        slots[tokens // 2] = -1
    slots = to_gpu(slots)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    q1 = q4.qk_norm_rope_append(q, k, v, pos, table, caches[0], slots, *w, eps=1e-5, interleaved=interleaved)
    q2, k2 = q4.qk_norm_rope(q, k, pos, table, *w, eps=1e-5, interleaved=interleaved)
    q4.paged_kv_append(k2, v, caches[1], slots)
    assert torch.equal(q1, q2)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name


def test_wrapper_refusals(q4):
    import torch

    x = torch.zeros((4, 4, 128), dtype=torch.float16, device="cuda")
    cache = q4.paged_kv_alloc(2, 16, 1, 128)
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = q4.rope_table(8, 128)
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    with pytest.raises(TypeError):
        q4.qk_norm_rope(q.float(), k, slots, table)
    with pytest.raises(TypeError):
        q4.qk_norm_rope(q, k, slots.long(), table)
    with pytest.raises(ValueError):
        q4.qk_norm_rope(q, k[:3], slots, table)
    with pytest.raises(ValueError):
        q4.qk_norm_rope(q, k, None, table)
    with pytest.raises(ValueError):
        q4.qk_norm_rope(x.transpose(1, 2), k, slots, table)
    with pytest.raises(ValueError):
        q4.paged_kv_append(q, q, cache, slots)
    with pytest.raises(ValueError):
        q4.paged_kv_append(k, v, cache, slots[:3])
    with pytest.raises(ValueError):
        q4.qk_norm_rope_append(q.cpu(), k, v, slots, table, cache, slots)
    with pytest.raises(q4.Q4Error):
        q4.paged_kv_alloc(2, 8, 1, 128)
    with pytest.raises(q4.Q4Error):
        q4.rope_table(8, 20)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_non_finite_groups(q4, bad):
    """A group that holds an infinity or a NaN reads back as NaN, the others are unharmed."""
    x = _qkv(4, 0, 2, 128, seed=21)
    x[1, 0, 40], x[2, 3, 127] = bad, bad
    cache = q4.paged_kv_alloc(1, 16, 2, 128, 32)
    slots = to_gpu(np.arange(4, dtype=np.int32))
    q4.paged_kv_append(to_gpu(x[:, :2]), to_gpu(x[:, 2:]), cache, slots)
    k, v = (to_np(t) for t in q4.paged_kv_dequant(cache, slots))
    clean = x.copy()
    clean[1, 0, 40] = clean[2, 3, 127] = 0
    want_k, want_v = (oracle.paged.store(clean[:, s], 32)[2] for s in (slice(0, 2), slice(2, 4)))
    want_k[1, 0, 32:64] = want_v[2, 1, 96:] = np.nan
    assert np.array_equal(k.astype(np.float64), want_k.astype(np.float16).astype(np.float64), equal_nan=True)
    assert np.array_equal(v.astype(np.float64), want_v.astype(np.float16).astype(np.float64), equal_nan=True)


def test_caches_made_by_hand(q4):
    """A cache's tensors are checked against its sizes, also in a copy with other fields."""
    import dataclasses

    import torch

    cache = q4.paged_kv_alloc(4, 32, 2, 128, 64)
    k = torch.randn((3, 2, 128), device="cuda").half()
    slots = torch.tensor([0, 40, 127], dtype=torch.int32, device="cuda")
    q4.paged_kv_append(k, k, cache, slots)
    same = dataclasses.replace(cache, k_codes=cache.k_codes.clone())
    assert all(torch.equal(a, b) for a, b in zip(q4.paged_kv_dequant(same, slots), q4.paged_kv_dequant(cache, slots)))
    wrong = [dict(page_size=64), dict(head_dim=256), dict(group=32), dict(v_codes=cache.v_codes[:3]),
             dict(k_scales=cache.k_scales[:, :1]), dict(v_scales=cache.v_scales[..., :32].contiguous()),
             dict(v_codes=cache.v_codes.transpose(0, 1)), dict(k_codes=cache.k_codes.view(-1))]
    for fields in wrong:
        with pytest.raises(ValueError):
            q4.paged_kv_append(k, k, dataclasses.replace(cache, **fields), slots)
    for fields in (dict(v_codes=cache.v_codes.view(torch.int8)), dict(k_scales=cache.k_scales.float())):
        with pytest.raises(TypeError):
            q4.paged_kv_append(k, k, dataclasses.replace(cache, **fields), slots)


def test_k_rounds_as_a_float64_array_converts(q4):
    """4097 rows, normed and turned: the bits of the float64 result as torch and numpy (through
    float32) convert it, on both sides of the few ties where rounding once would differ."""
    import torch

    x = _qkv(4097, 1, 8, 128, seed=77)
    w = (1 + 0.3 * np.random.default_rng(3).standard_normal(128)).astype(np.float16)
    pos, table = np.arange(4097, dtype=np.int32), _table(4097, 64)
    g = to_gpu(x)
    _, k = q4.qk_norm_rope(g[:, :1], g[:, 1:9], to_gpu(pos), to_gpu(table), to_gpu(w), to_gpu(w), 1e-6, True)
    ref = oracle.paged.norm_rope(x[:, 1:9], w, 1e-6, table[:, :, 0], table[:, :, 1], True)
    want = ref.astype(np.float32).astype(np.float16)
    assert np.array_equal(torch.from_numpy(ref).half().numpy().view(np.uint16), want.view(np.uint16))
    assert (want != ref.astype(np.float16)).any()
    assert _same_bits(to_np(k), want)


def _norm_rope_ref(x, weight, eps, table, pos, interleaved):
    """The formula in float64 with the arithmetic of infinities (0 * infinity is NaN)."""
    cos, sin = (None, None) if table is None else (table[pos, :, 0], table[pos, :, 1])
    with np.errstate(invalid="ignore"):
        return oracle.paged.norm_rope(x, weight, eps, cos, sin, interleaved)


def _equal_q(got, ref):
    """q against the formula: NaN and infinities exactly, the rest within half a float16 step and 16
    roundings of float32 (2^-24 each of the two terms of a channel, together below 64 in size here)."""
    got = got.astype(np.float64)
    with np.errstate(over="ignore"):
        want = ref.astype(np.float16).astype(np.float64)
    odd = ~np.isfinite(want)
    assert np.array_equal(np.where(odd, got, 0), np.where(odd, want, 0), equal_nan=True)
    err = np.abs(np.where(odd, 0, got) - np.where(odd, 0, ref))
    assert np.all(err <= 2.0 ** -11 * np.abs(np.where(odd, 0, ref)) + 2.0 ** -25 + 16 * 2.0 ** -24 * 64), err.max()


@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (64, True), (128, False), (128, True)])
def test_infinities_in_q(q4, rot, interleaved):
    """An infinity in q stays where the formula puts it: without a rotation and behind rot_dim it is
    itself, inside it reaches its pair."""
    x = np.random.default_rng(rot).standard_normal((6, 4, 128)).astype(np.float16)
    x[1, 0, 3], x[2, 1, 70], x[3, 2, 127], x[4, 3, 100], x[5, 0, 64] = np.inf, -np.inf, np.inf, -np.inf, np.nan
    pos = np.array([1, 2, 3, 4, 5, 6], np.int32)
    table = _table(8, rot) if rot else None
    g = to_gpu(x)
    q, _ = q4.qk_norm_rope(g, g[:, :1], to_gpu(pos) if rot else None, to_gpu(table) if rot else None,
                           interleaved=interleaved)
    _equal_q(to_np(q), _norm_rope_ref(x, None, 0.0, table, pos, interleaved))


@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (64, True), (128, False), (128, True)])
def test_infinities_under_a_norm(q4, rot, interleaved):
    """One infinity makes its head's mean square infinite: its channel (and pair) NaN, the others zero, in
    q, in k and in the cache, where only the groups that hold a NaN read back as NaN."""
    import torch

    r = np.random.default_rng(rot + 1)
    x = r.standard_normal((5, 8, 128)).astype(np.float16)
    x[1, [0, 4, 6], 3], x[2, [1, 5, 7], 70], x[3, [2, 4, 6], 127] = np.inf, -np.inf, np.inf
    w = [(1 + 0.3 * r.standard_normal(128)).astype(np.float16) for _ in range(2)]
    pos = np.array([1, 2, 3, 4, 5], np.int32)
    table = _table(8, rot) if rot else None
    g = to_gpu(x)
    rest = (to_gpu(pos) if rot else None, to_gpu(table) if rot else None)
    q, k = q4.qk_norm_rope(g[:, :4], g[:, 4:6], *rest, to_gpu(w[0]), to_gpu(w[1]), 1e-6, interleaved)
    ref_q = _norm_rope_ref(x[:, :4], w[0], 1e-6, table, pos, interleaved)
    ref_k = _norm_rope_ref(x[:, 4:6], w[1], 1e-6, table, pos, interleaved)
    assert np.isnan(ref_k).any() and (ref_k == 0).any()
    _equal_q(to_np(q), ref_q)
    want_k = ref_k.astype(np.float32).astype(np.float16)
    assert np.array_equal(to_np(k), want_k, equal_nan=True)
    cache = q4.paged_kv_alloc(1, 16, 2, 128, 32)
    slots = to_gpu(np.arange(5, dtype=np.int32))
    q2 = q4.qk_norm_rope_append(g[:, :4], g[:, 4:6], g[:, 6:], *rest, cache, slots, to_gpu(w[0]), to_gpu(w[1]), 1e-6,
                                interleaved)
    assert np.array_equal(to_np(q2), to_np(q), equal_nan=True)
    for got, rows in zip(q4.paged_kv_dequant(cache, slots), (want_k, x[:, 6:])):
        bad = ~np.isfinite(rows.reshape(5, 2, 4, 32)).all(-1)
        want = oracle.paged.store(np.where(np.repeat(bad, 32, -1), np.float16(0), rows), 32)[2].astype(np.float16)
        want[np.repeat(bad, 32, -1)] = np.nan
        assert bad.any() and not bad.all()
        assert np.array_equal(to_np(got), want, equal_nan=True)
    assert torch.isfinite(q4.paged_kv_dequant(cache, slots)[0][[0, 4]]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinite_weight_behind_the_rotation(q4, interleaved):
    """An infinite norm weight of a channel that is not turned gives that channel infinities only."""
    x = np.random.default_rng(5).standard_normal((3, 4, 128)).astype(np.float16)
    w = np.ones(128, np.float16)
    w[100] = np.inf
    pos, table = np.array([1, 2, 3], np.int32), _table(8, 64)
    g = to_gpu(x)
    q, k = q4.qk_norm_rope(g[:, :2], g[:, 2:], to_gpu(pos), to_gpu(table), to_gpu(w), to_gpu(w), 1e-6, interleaved)
    ref = _norm_rope_ref(x, w, 1e-6, table, pos, interleaved)
    assert np.isinf(ref[..., 100]).all() and np.isfinite(np.delete(ref, 100, -1)).all()
    _equal_q(to_np(q), ref[:, :2])
    assert np.array_equal(to_np(k), ref[:, 2:].astype(np.float32).astype(np.float16))


def test_copies_and_pickles_of_a_used_cache(q4):
    """A cache that has been used copies and pickles as an unused one does, and the copies work."""
    import copy
    import io
    import pickle

    import torch

    cache = q4.paged_kv_alloc(3, 16, 2, 128, 64)
    k = torch.randn((5, 2, 128), device="cuda").half()
    slots = torch.tensor([0, 40, 17, 3, 22], dtype=torch.int32, device="cuda")
    q4.paged_kv_append(k, k, cache, slots)
    want = q4.paged_kv_dequant(cache, slots)
    deep = copy.deepcopy(cache)
    file = io.BytesIO()
    torch.save(cache, file)
    file.seek(0)
    for other in (copy.copy(cache), deep, pickle.loads(pickle.dumps(cache)), torch.load(file, weights_only=False)):
        assert all(torch.equal(a, b) for a, b in zip(q4.paged_kv_dequant(other, slots), want))
    assert deep.k_codes.data_ptr() != cache.k_codes.data_ptr()
    q4.paged_kv_append(-k, -k, deep, slots)
    assert all(torch.equal(a, b) for a, b in zip(q4.paged_kv_dequant(cache, slots), want))


def test_norm_of_subnormal_rows(q4):
    """Rows among float16's subnormals (all below 2^-14) keep their mean square."""
    r = np.random.default_rng(9)
    x = (r.standard_normal((4, 3, 128)) * 2.0 ** -17).astype(np.float16)
    w = np.ones(128, np.float16)
    g = to_gpu(x)
    q, k = q4.qk_norm_rope(g[:, :2], g[:, 2:], None, None, to_gpu(w), to_gpu(w), 1e-14)
    ref = _norm_rope_ref(x, w, np.float64(np.float32(1e-14)), None, None, False)
    assert np.abs(ref).max() > 1
    _equal_q(to_np(q), ref[:, :2])
    assert _same_bits(to_np(k), ref[:, 2:].astype(np.float32).astype(np.float16))


def test_far_slots_and_rows(q4):
    """Slots, rows and tokens whose offsets pass 32 bits: a cache of 8 GiB of codes for K and as many for
    V, rows 2^30 elements apart; the same bits as near ones."""
    import torch

    say("far slots and rows")
    pages, page, heads, d = (1 << 18) + 64, 64, 8, 128
    far = q4.paged_kv_alloc(pages, page, heads, d, 128)
    near = q4.paged_kv_alloc(4, page, heads, d, 128)
    n, hq = 150, 16
    r = np.random.default_rng(11)
    k, v = (to_gpu(r.standard_normal((n, heads, d)).astype(np.float16)) for _ in range(2))
    t = np.arange(n)
    table = np.array([[pages - 1, pages - 7, pages // 2]], np.int32)
    slots = [to_gpu((tab[0][t // page] * page + t % page).astype(np.int32)) for tab in (table, np.array([[2, 0, 3]]))]
    for cache, s in zip((far, near), slots):
        q4.paged_kv_append(k, v, cache, s)
    for a, b in zip(q4.paged_kv_dequant(far, slots[0]), q4.paged_kv_dequant(near, slots[1])):
        assert torch.equal(a, b) and bool(a.any())
    rest = (to_gpu(np.array([0, 3], np.int32)), to_gpu(np.array([n], np.int32)), 3, n)
    q = to_gpu(r.standard_normal((3, hq, d)).astype(np.float16))
    want = q4.paged_attention(q, near, to_gpu(np.array([[2, 0, 3]], np.int32)), *rest)
    wide = torch.zeros((2 << 30) + hq * d, dtype=torch.float16, device="cuda").as_strided((3, hq, d), (1 << 30, d, 1))
    wide.copy_(q)
    assert torch.equal(q4.paged_attention(wide, far, to_gpu(table), *rest), want)
    pos, turn = to_gpu(np.array([5, 6, 7], np.int32)), q4.rope_table(16, d)
    a, _ = q4.qk_norm_rope(q, k[:3], pos, turn)
    b, _ = q4.qk_norm_rope(wide, k[:3], pos, turn, q_out=wide)
    assert torch.equal(a, b)
