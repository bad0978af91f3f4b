"""The serving operators (appending to the paged cache, decode attention) against
plain implementations in 64 bits.

Tolerances.  u(t) = torch.finfo(t).eps / 2 is the relative rounding of type t
(bf16 2^-8, E4M3 2^-4).  An appended value is computed in fp32 and rounded
once: it is within u of its exact value, plus the fp32 error of a 512-term sum,
a square root and three products (below 2^-18 relative, and 2^-20 absolute for
a rotated pair whose terms cancel, times its length).

Decode rounds the absorbed query, the rotated q_rope, the softmax weights, the
latent state before W_UV and the output to bf16 (or to something finer).
 - A score s_t = scale (qlat . c_t + qrot . k_t) is a sum of 576 terms, each off
   by an independent relative error of at most u, standard deviation u / sqrt(3)
   at most.  lse moves by no more than the largest score error: six standard
   deviations of it, 6 scale u / sqrt(3) max_t sqrt(sum (qlat c_t)^2 + (qrot k_t)^2),
   bound lse (plus 2^-15 for the exponentials and sums in fp32).
 - The output takes five roundings of standard deviation u / sqrt(3) = 2.3e-3
   at most (scores, through their unit-size logits; weights; state; output; and
   the query's through the keys' common direction): 5.1e-3 of the output's norm
   together, held to twice that.
   (The weights of an FP8 cache are sums of two E5M2 terms, within 2^-7: 2^-7 /
   sqrt(3) in the place of one u / sqrt(3), 6.4e-3 together, under the same bound.)
"""
import ctypes
import math

import numpy as np
import pytest

from mla_prefix_cache_gb300 import _lib, workload as W

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu

U_BF16 = torch.finfo(torch.bfloat16).eps / 2
U_E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2
REL_RMS = 1.02e-2


@pytest.fixture(scope="module")
def api():
    from mla_prefix_cache_gb300 import api as A
    _lib.load()
    return A


# ------------------------------------------------------------------ 64-bit references

def angles(pos, theta=10000.0):
    return np.asarray(pos, dtype=np.float64)[..., None] * theta ** (-2.0 * np.arange(32) / 64)


def turn(x, a):
    """Pairs (2k, 2k+1) of x's last axis turned by a."""
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * a)
    return np.stack((z.real, z.imag), -1).reshape(x.shape)


def bf16_values(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def cache_values(rows, kv_dtype, kv_scale):
    """(c, k_rope) of cached rows in 64 bits."""
    if kv_dtype == "bf16":
        v = bf16_values(rows)
        return v[..., :512], v[..., 512:]
    codes = torch.from_numpy(np.ascontiguousarray(rows[..., :512])).view(torch.float8_e4m3fn).double().numpy()
    return codes * kv_scale, bf16_values(np.ascontiguousarray(rows[..., 512:]).view(np.uint16))


def ranges_of(segs, n):
    """(start, stop, rope offset) of a request's visible keys."""
    if segs is None:
        return [(0, n, 0)]
    end, out = 0, []
    for s, length, off in segs:
        lo = min(max(s, end), n)
        hi = max(lo, min(s + max(length, 0), n))
        out.append((lo, hi, off))
        end = hi
    return out + [(min(end, n), n, 0)]


def decode_ref(wl, lens=None, cu=None, segs=None):
    """(out, lse, lse tolerance) of every row a request has, NaN elsewhere.  segs: per request, or None."""
    lens = wl.seq_lens if lens is None else lens
    cu = wl.cu_q if cu is None else cu
    T, H = wl.q.shape[0], wl.num_heads
    out, lse, tol = np.full((T, H, 128), np.nan), np.full((T, H), np.nan), np.zeros((T, H))
    q, w = bf16_values(wl.q), bf16_values(wl.kv_b_proj)
    wk, wv = w[:, :H * 128].reshape(512, H, 128), w[:, H * 128:].reshape(512, H, 128)
    for r in range(len(lens)):
        n, E = int(lens[r]), int(cu[r + 1] - cu[r])
        t = np.arange(n)
        c, k = cache_values(wl.kv_cache[wl.block_table[r][t // 64], t % 64], wl.kv_dtype, wl.kv_scale)
        for i in range(E):
            row = int(cu[r]) + i
            lat = np.einsum("hd,chd->hc", q[row, :, :128], wk)
            s, v, var = [], [], []
            for lo, hi, off in ranges_of(None if segs is None else segs[r], n):
                hi = min(hi, n - E + i + 1)
                if hi <= lo:
                    continue
                rot = turn(q[row, :, 128:], angles(int(wl.q_pos[row]) - off, wl.rope_theta))
                s.append(wl.softmax_scale * (lat @ c[lo:hi].T + rot @ k[lo:hi].T))
                var.append((lat ** 2) @ (c[lo:hi] ** 2).T + (rot ** 2) @ (k[lo:hi] ** 2).T)
                v.append(c[lo:hi])
            if not s:
                out[row], lse[row] = 0.0, -np.inf
                continue
            s, v, var = np.concatenate(s, 1), np.concatenate(v), np.concatenate(var, 1)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            lse[row] = m[:, 0] + np.log(p.sum(1))
            out[row] = np.einsum("hc,chd->hd", (p / p.sum(1, keepdims=True)) @ v, wv)
            tol[row] = 6 * abs(wl.softmax_scale) * U_BF16 / math.sqrt(3) * np.sqrt(var.max(1)) + 2.0 ** -15
    return out, lse, tol


def assert_decode(out, lse, ref):
    out, ref_out, ref_lse, tol = out.double().cpu().numpy(), *ref
    rows = ~np.isnan(ref_lse[:, 0])
    assert np.isfinite(out[rows]).all(), "non-finite output"
    empty = np.isneginf(ref_lse)
    assert (out[empty] == 0).all(), "a row without keys is not 0"
    d = out[rows] - ref_out[rows]
    den = math.sqrt(float((ref_out[rows] ** 2).mean()))
    rel = math.sqrt(float((d ** 2).mean())) / den if den else float(np.abs(d).max(initial=0.0))
    assert rel <= REL_RMS, f"rel rms {rel:.3e}"
    # no row hides a fault in the mean over all: a row's own error, six times the mean's share of 128 values
    row_rel = np.sqrt((d ** 2).mean(-1)) / np.maximum(np.sqrt((ref_out[rows] ** 2).mean(-1)), 1e-3 * den)
    live = ~empty[rows]
    assert (row_rel[live] <= 6 * REL_RMS).all(), f"a row's rel rms {row_rel[live].max():.3e}"
    if lse is not None:
        lse = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(lse[rows]), empty[rows]), "rows without keys differ"
        fin = rows[:, None] & ~empty
        e = np.abs(lse[fin] - ref_lse[fin])
        assert (e <= tol[fin]).all(), f"lse off by {e.max():.3e}, {(e / tol[fin]).max():.2f} of its bound"


def seg_tensors(segs):
    """(segments, seg_ptr) device tensors of per-request lists."""
    ptr = np.cumsum([0] + [len(s) for s in segs]).astype(np.int32)
    flat = np.asarray([x for s in segs for x in s], dtype=np.int64).reshape(-1, 3)
    return torch.from_numpy(flat).cuda(), torch.from_numpy(ptr).cuda()


class Dev:
    """Device copies of a workload for the serving calls."""

    def __init__(self, api, wl, segs=None):
        d = api.DeviceWorkload(wl)
        self.api, self.wl = api, wl
        self.q, self.q_pos, self.kv_cache, self.block_table, self.kv_b_proj = d.q, d.q_pos, d.kv_cache, d.block_table, d.kv_b_proj
        self.seq_lens = torch.from_numpy(wl.seq_lens).cuda()
        self.cu_q = torch.from_numpy(wl.cu_q).cuda()
        self.segments, self.seg_ptr = (None, None) if segs is None else seg_tensors(segs)

    def decode(self, **kw):
        a = dict(softmax_scale=self.wl.softmax_scale, rope_theta=self.wl.rope_theta, kv_scale=self.wl.kv_scale,
                 cu_q=self.cu_q, segments=self.segments, seg_ptr=self.seg_ptr, return_lse=True)
        a.update(kw)
        return self.api.decode(self.q, self.q_pos, self.kv_cache, self.block_table, self.seq_lens, self.kv_b_proj, **a)


def check_decode(api, wl, segs=None, **kw):
    d = Dev(api, wl, segs)
    out, lse = d.decode(**kw)
    assert api.device_error(api.decode.last_workspace) == 0
    assert_decode(out, lse, decode_ref(wl, segs=segs))
    return d, out, lse


# ------------------------------------------------------------------ host checks

@pytest.fixture(scope="module")
def lib():
    from mla_prefix_cache_gb300 import build
    import os
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def test_append_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)

    def call(kv=d, stride=576, pos=d, w=d, eps=1e-6, cu=d, sl=d, B=2, rows=5, bt=d, mb=4, theta=1e4, cache=d, kvt=0,
             scale=1.0, nb=8):
        return lib.mla_cache_append(kv, stride, pos, w, eps, cu, sl, B, rows, bt, mb, theta, cache, kvt, scale, nb,
                                    None, None)
    bad = [dict(kv=None), dict(kv=ctypes.c_void_p(4104)), dict(stride=575), dict(stride=580), dict(stride=-576),
           dict(pos=None), dict(w=ctypes.c_void_p(4098)), dict(eps=-1.0), dict(eps=float("nan")),
           dict(eps=float("inf")), dict(cu=None), dict(sl=None), dict(B=0), dict(B=-1), dict(rows=-1), dict(bt=None),
           dict(mb=0), dict(mb=1 << 26), dict(theta=1.0), dict(theta=float("nan")), dict(cache=None),
           dict(cache=ctypes.c_void_p(4104)), dict(kvt=2), dict(nb=0), dict(kvt=1, scale=0.0),
           dict(kvt=1, scale=float("nan")), dict(kvt=1, scale=1e-39)]      # (whose reciprocal overflows)
    for b in bad:
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(rows=0, kv=None, pos=None) == _lib.MLA_OK      # nothing to do
    assert call(rows=0, B=0, cu=None) == _lib.MLA_OK


def test_decode_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)
    n = lib.mla_decode_workspace_size(2, 5, 8)
    assert n >= 256
    assert lib.mla_decode_workspace_size(2, 5, 0) == 0 and lib.mla_decode_workspace_size(2, 5, 129) == 0
    assert lib.mla_decode_workspace_size(-1, 5, 8) == 0 and lib.mla_decode_workspace_size(2, -1, 8) == 0

    def call(q=d, pos=d, cache=d, kvt=0, scale=1.0, nb=8, bt=d, mb=4, sl=d, cu=d, B=2, T=5, H=8, sg=None, sp=None,
             ns=0, w=d, sm=0.07, theta=1e4, out=d, od=0, ws=d, wb=n):
        return lib.mla_decode(q, pos, cache, kvt, scale, nb, bt, mb, sl, cu, B, T, H, sg, sp, ns, w, sm, theta, out,
                              od, None, ws, wb, None)
    bad = [dict(q=None), dict(q=ctypes.c_void_p(4104)), dict(pos=None), dict(cache=None), dict(kvt=5), dict(nb=0),
           dict(bt=None), dict(mb=0), dict(sl=None), dict(cu=None), dict(B=0), dict(B=-2), dict(T=-1), dict(H=0),
           dict(sg=d), dict(sp=d), dict(ns=-1), dict(w=None), dict(w=ctypes.c_void_p(4098)), dict(sm=float("nan")), dict(sm=0.0), dict(sm=-0.1),
           dict(theta=0.5), dict(out=None), dict(out=ctypes.c_void_p(4104)), dict(od=2), dict(kvt=1, scale=-1.0)]
    for b in bad:
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(H=129) == _lib.MLA_ERR_UNSUPPORTED
    assert call(kvt=1, scale=2.0 ** -33) == call(kvt=1, scale=2.0 ** 33) == _lib.MLA_ERR_UNSUPPORTED
    assert call(nb=1 << 25) == _lib.MLA_ERR_UNSUPPORTED            # 2^31 cached tokens
    assert call(T=1 << 24, H=64) == _lib.MLA_ERR_UNSUPPORTED       # 2^30 rows
    assert call(mb=1 << 24, T=1 << 15, H=128) == _lib.MLA_ERR_UNSUPPORTED     # 2^15 items of 2^23 tiles
    for b in (dict(ws=None), dict(ws=ctypes.c_void_p(4104)), dict(wb=n - 1)):
        assert call(**b) == _lib.MLA_ERR_WORKSPACE, b
    assert call(T=0, q=None) == _lib.MLA_OK


def test_reference_ranges_cut_segments():
    assert ranges_of(None, 9) == [(0, 9, 0)]
    assert ranges_of([(0, 4, 0), (2, 4, 7), (20, 5, 3)], 12) == [(0, 4, 0), (4, 6, 7), (12, 12, 3), (12, 12, 0)]
    assert ranges_of([(1, -3, 5)], 6) == [(1, 1, 5), (1, 6, 0)]


# ------------------------------------------------------------------ append

def append_case(lens, new, kv_dtype, *, norm=True, stride=576, seed=0, extra_rows=0, pos_scale=1, theta=10000.0):
    rng = np.random.Generator(np.random.PCG64(seed))
    rows = sum(new) + extra_rows
    need = [-(-n // 64) for n in lens]
    pool = sum(need) + 3
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    kv = W.f32_to_bf16_bits(3.0 * rng.standard_normal((rows, stride), dtype=np.float32))
    weight = W.f32_to_bf16_bits(1.0 + 0.3 * rng.standard_normal(512, dtype=np.float32)) if norm else None
    pos = np.concatenate([np.arange(n - e, n) for n, e in zip(lens, new)] + [np.zeros(extra_rows)]).astype(np.int64) * pos_scale
    cache = rng.integers(0, 120, (pool, 64, 1152 if kv_dtype == "bf16" else 640), dtype=np.uint8)
    return dict(kv=kv, weight=weight, pos=pos.astype(np.int32), cache=cache, table=table, theta=theta,
                lens=np.asarray(lens, dtype=np.int32), cu=np.cumsum([0] + list(new)).astype(np.int32), kv_dtype=kv_dtype,
                scale=1.0 if kv_dtype == "bf16" else 0.0137)


def append_ref(c):
    """{(block, slot): (c, k)} of the rows that are written, in 64 bits (c unscaled)."""
    x = bf16_values(c["kv"][:, -576:])
    out = {}
    for r, n in enumerate(c["lens"]):
        for row in range(c["cu"][r], c["cu"][r + 1]):
            t = int(n) - (int(c["cu"][r + 1]) - row)
            if t < 0:
                continue
            lat = x[row, :512]
            if c["weight"] is not None:
                lat = lat / np.sqrt((lat ** 2).mean() + 1e-6) * bf16_values(c["weight"])
            out[int(c["table"][r, t // 64]), t % 64] = lat, turn(x[row, 512:], angles(int(c["pos"][row]), c["theta"]))
    return out


def run_append(api, c, uniform=False, cu=None, dev_error=None, stream=None):
    kv = torch.from_numpy(c["kv"].view(np.int16)).cuda().view(torch.bfloat16)[:, -576:]
    cache = torch.from_numpy(c["cache"].copy()).cuda()
    if c["kv_dtype"] == "bf16":
        cache = cache.view(torch.bfloat16)
    w = None if c["weight"] is None else torch.from_numpy(c["weight"].view(np.int16)).cuda().view(torch.bfloat16)
    cuq = None if uniform else torch.from_numpy(c["cu"]).cuda()
    api.cache_append(kv, torch.from_numpy(c["pos"]).cuda(), cache, torch.from_numpy(c["table"]).cuda(),
                     torch.from_numpy(c["lens"]).cuda(), cu_q=cuq, norm_weight=w, rope_theta=c["theta"],
                     kv_scale=c["scale"], dev_error=dev_error, stream=stream)
    return cache


def check_append(c, cache, ref=None):
    ref = append_ref(c) if ref is None else ref
    got = cache.view(torch.uint8).cpu().numpy()
    untouched = np.ones(got.shape[:2], dtype=bool)
    for (b, s), (lat, k) in ref.items():
        untouched[b, s] = False
        if c["kv_dtype"] == "bf16":
            v = bf16_values(np.ascontiguousarray(got[b, s]).view(np.uint16))
            assert (np.abs(v[:512] - lat) <= (U_BF16 + 2.0 ** -18) * np.abs(lat)).all()
            rope = v[512:]
        else:
            v = torch.from_numpy(np.ascontiguousarray(got[b, s, :512])).view(torch.float8_e4m3fn).double().numpy()
            want = np.clip(lat / c["scale"], -448, 448)
            # half a step: 2^-4 of a normal value, 2^-10 below the smallest normal (2^-6)
            assert (np.abs(v - want) <= np.maximum(U_E4M3 * np.abs(want), 2.0 ** -10) * (1 + 2.0 ** -12)).all()
            rope = bf16_values(np.ascontiguousarray(got[b, s, 512:]).view(np.uint16))
        length = np.repeat(np.sqrt(k[0::2] ** 2 + k[1::2] ** 2), 2)
        assert (np.abs(rope - k) <= U_BF16 * np.abs(k) + 2.0 ** -20 * length).all()
    assert np.array_equal(got[untouched], c["cache"][untouched]), "another row of the cache changed"


APPEND = [
    dict(lens=[1], new=[1]),                                          # a first token
    dict(lens=[130, 64, 65, 1, 700], new=[3, 64, 65, 1, 257]),        # ragged, blocks begun and filled
    dict(lens=[200] * 40, new=[1] * 40),                              # a decode step
    dict(lens=[90, 0, 70, 5], new=[2, 0, 0, 5]),                      # requests without rows
    dict(lens=[1000], new=[1000], pos_scale=1031, theta=500000.0),    # far positions
]


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("case", APPEND, ids=["one", "ragged", "step", "empty", "far"])
def test_append_matches_64_bits(api, case, norm, kv):
    c = append_case(**case, kv_dtype=kv, norm=norm, seed=len(case["lens"]))
    check_append(c, run_append(api, c))


@gpu
@pytest.mark.parametrize("reqs", [31, 32, 33, 1000, 1025, 1100])
def test_append_finds_the_request_of_every_row(api, reqs):
    # around 32 and 1024 requests the search takes another round; every third request has no rows
    new = [(r * 7) % 3 for r in range(reqs)]
    c = append_case([5 + n for n in new], new, "fp8_e4m3", seed=reqs)
    check_append(c, run_append(api, c))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_append_strided_rows_uniform_batch(api, kv):
    c = append_case([66, 3, 129], [3, 3, 3], kv, stride=2112, seed=3)
    check_append(c, run_append(api, c, uniform=True))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_append_leaves_padding_out(api, kv):
    # a padded request (length 0 with one row), a row of negative token index, rows behind the last request
    c = append_case([70, 66, 2], [1, 1, 2], kv, seed=4, extra_rows=5)
    c["lens"] = np.asarray([70, 0, 1], dtype=np.int32)
    check_append(c, run_append(api, c))


@gpu
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 5])
def test_append_bad_block_is_reported_and_nothing_written(api, bad):
    c = append_case([130, 64], [2, 1], "bf16", seed=5)
    c["lens"] = np.asarray([130, 64], dtype=np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = append_ref(c)
    if bad == 5:      # a token behind the block table
        ref.pop((int(c["table"][1, 0]), 63))
        c["lens"][1] = 64 * c["table"].shape[1] + 1
    else:
        for s in (0, 1):
            ref.pop((int(c["table"][0, 2]), s))
        c["table"][0, 2] = bad
    check_append(c, run_append(api, c, dev_error=err), ref)
    assert int(err.item()) == 1


@gpu
def test_append_leaves_rows_before_the_first_request_out(api):
    c = append_case([70, 66], [2, 3], "bf16", seed=9, extra_rows=4)
    c["kv"], c["pos"], c["cu"] = np.roll(c["kv"], 2, 0), np.roll(c["pos"], 2), c["cu"] + 2
    check_append(c, run_append(api, c))


@gpu
def test_append_saturates_and_keeps_infinities_to_themselves(api):
    c = append_case([3], [3], "fp8_e4m3", norm=False, seed=6)
    x = bf16_values(c["kv"])
    x[1, :4] = [1e30, -1e30, np.inf, -np.inf]
    x[1, 4] = np.nan
    c["kv"] = W.f32_to_bf16_bits(x.astype(np.float32))
    got = run_append(api, c).cpu().numpy()
    b = int(c["table"][0, 0])
    assert got[b, 1, :4].tolist() == [0x7E, 0xFE, 0x7E, 0xFE] and got[b, 1, 4] & 0x7F == 0x7F
    c["kv"][1] = c["kv"][0]
    ref = append_ref(c)
    ref.pop((b, 1))
    c["cache"][b, 1] = got[b, 1]
    check_append(c, torch.from_numpy(got), ref)


@gpu
def test_append_far_into_a_large_pool(api):
    # byte offsets past 2^32
    nb = (1 << 32) // (64 * 1152) + 200
    cache = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    c = append_case([3], [3], "bf16", seed=8)
    c["table"][0, 0] = nb - 1
    kv = torch.from_numpy(c["kv"].view(np.int16)).cuda().view(torch.bfloat16)
    w = torch.from_numpy(c["weight"].view(np.int16)).cuda().view(torch.bfloat16)
    api.cache_append(kv, torch.from_numpy(c["pos"]).cuda(), cache, torch.from_numpy(c["table"]).cuda(),
                     torch.from_numpy(c["lens"]).cuda(), norm_weight=w)
    assert int((cache[:-1] != 0).sum()) == 0
    c["cache"] = np.zeros((1, 64, 1152), dtype=np.uint8)
    check_append(c, cache[-1:], {(0, s): v for (_, s), v in append_ref(c).items()})


@gpu
def test_append_refusals(api):
    c = append_case([70, 66], [1, 1], "bf16", seed=7)
    kv = torch.from_numpy(c["kv"].view(np.int16)).cuda().view(torch.bfloat16)
    args = dict(pos=torch.from_numpy(c["pos"]).cuda(), kv_cache=torch.from_numpy(c["cache"]).cuda().view(torch.bfloat16),
                block_table=torch.from_numpy(c["table"]).cuda(), seq_lens=torch.from_numpy(c["lens"]).cuda())
    for kw in (dict(kv=kv.cpu()), dict(kv=kv.float()), dict(kv=kv[:, :560]), dict(kv=kv.t().contiguous().t()),
               dict(kv=torch.zeros((2, 580), dtype=torch.bfloat16, device="cuda")[:, :576]),
               dict(pos=args["pos"][:1]), dict(pos=args["pos"].long()), dict(seq_lens=args["seq_lens"].cpu()),
               dict(seq_lens=args["seq_lens"].long()), dict(block_table=args["block_table"][:1]),
               dict(cu_q=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(kv_cache=args["kv_cache"].half()),
               dict(norm_weight=torch.ones(511, dtype=torch.bfloat16, device="cuda")),
               dict(norm_weight=torch.ones(512, device="cuda")), dict(kv=kv[:1].expand(3, 576), pos=args["pos"][:1].expand(3))):
        with pytest.raises((ValueError, _lib.MLAError)):
            api.cache_append(**{**args, "kv": kv, **kw})
    assert np.array_equal(args["kv_cache"].view(torch.uint8).cpu().numpy(), c["cache"])
    api.cache_append(kv[:0], args["pos"][:0], *[args[k] for k in ("kv_cache", "block_table", "seq_lens")])   # no rows


# ------------------------------------------------------------------ decode

DECODE = [
    ("one_key", 128, [0], [1]),
    ("short", 128, [499], [1]),
    ("heads_odd", 5, [63, 64, 65, 127, 0, 300], [1, 1, 1, 1, 1, 1]),
    ("one_head", 1, [200, 1000], [1, 1]),
    ("tile_edges", 16, [126, 127, 128, 129, 191, 192, 255, 256], [1, 1, 1, 1, 1, 1, 1, 1]),
    ("few_queries", 40, [130, 0, 517], [3, 4, 2]),
    ("row_tiles", 128, [300, 77], [4, 1]),
    ("ragged_rows", 33, [61, 190, 0, 1000, 5], [1, 9, 2, 4, 7]),
    ("long", 16, [9000], [2]),
    ("many", 3, [(37 * i) % 211 for i in range(150)], [1 + i % 2 for i in range(150)]),
    ("wide", 128, [60 + (29 * i) % 200 for i in range(70)], [1] * 70),       # 64 tokens of a head a CTA at the end
    ("mid", 64, [200 + i for i in range(25)], [2] * 25),                      # 32
]


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", DECODE, ids=[c[0] for c in DECODE])
def test_decode_matches_64_bits(api, case, kv):
    name, H, ctx, ext = case
    check_decode(api, W.make_workload(name, H, ctx, ext, kv_dtype=kv, seed=len(ctx) + H))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_uniform_batch_bf16_out_without_lse(api, kv):
    wl = W.make_workload("u", 24, [100, 400, 1], [2, 2, 2], kv_dtype=kv, seed=31)
    d = Dev(api, wl)
    out = d.decode(cu_q=None, return_lse=False, out_dtype=torch.bfloat16)
    assert out.dtype == torch.bfloat16
    assert_decode(out, None, decode_ref(wl))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_documents(api, kv):
    # documents at canonical positions; one request without any, one whose documents leave keys out,
    # overlap and reach behind the sequence; hidden keys hold NaN
    wl = W.make_workload("d", 16, [600, 300, 513, 64], [2, 1, 3, 1], kv_dtype=kv, seed=32)
    segs = [[(0, 200, 0), (200, 200, 200), (400, 200, 400)], [], [(7, 100, 7), (120, 129, 100), (200, 150, 180)],
            [(0, 30, 0), (40, 10 ** 12, 17)]]
    for r in range(4):
        seen = np.zeros(int(wl.seq_lens[r]), dtype=bool)
        for lo, hi, _ in ranges_of(segs[r], int(wl.seq_lens[r])):
            seen[lo:hi] = True
        for t in np.flatnonzero(~seen):
            wl.kv_cache[wl.block_table[r][t // 64], t % 64] = W.BF16_NAN if kv == "bf16" else W.E4M3_NAN
    check_decode(api, wl, segs)
    # no segments listed at all: every key, offset 0
    wl2 = W.make_workload("d2", 16, [600, 300], [2, 1], kv_dtype=kv, seed=33)
    check_decode(api, wl2, [[], []])


@gpu
def test_decode_documents_many_offsets(api):
    segs = [[(17 * i, 17, 10 ** 6 + 1000 * i) for i in range(60)]]
    check_decode(api, W.make_workload("dm", 20, [1100], [2], seed=34), segs)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_peaked_rows(api, kv):
    # logits of standard deviation 4: rows rest on few keys, and their maximum rises late
    wl = W.make_workload("p", 16, [1500, 700], [1, 2], kv_dtype=kv, seed=35)
    wl.q = W.f32_to_bf16_bits((4.0 * bf16_values(wl.q)).astype(np.float32))
    d = Dev(api, wl)
    out, lse = d.decode()
    ref = decode_ref(wl)
    _, ref_lse, tol = ref
    e = np.abs(lse.double().cpu().numpy() - ref_lse)
    assert (e <= tol).all()
    # a score error of four times the size goes into the weights: the bound grows with it
    rel = np.linalg.norm(out.double().cpu().numpy() - ref[0]) / np.linalg.norm(ref[0])
    assert rel <= 4 * REL_RMS


@gpu
def test_decode_empty_rows(api):
    # a request of length 0, one shorter than its rows, a live one between them
    wl = W.make_workload("e", 16, [0, 90, 0], [2, 1, 4], seed=36)
    lens = np.asarray([0, 91, 2], dtype=np.int32)
    d = Dev(api, wl)
    d.seq_lens = torch.from_numpy(lens).cuda()
    out, lse = d.decode()
    assert api.device_error(api.decode.last_workspace) == 0
    ref = decode_ref(wl, lens=lens)
    assert np.isneginf(ref[1][[0, 1, 3, 4]]).all() and np.isfinite(ref[1][[2, 5, 6]]).all()
    assert_decode(out, lse, ref)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_more_requests_than_threads(api, kv):
    # over 512 requests a thread of the schedule takes several; requests without rows or keys among them
    n = 1100
    check_decode(api, W.make_workload("mr", 2, [(13 * i) % 70 for i in range(n)], [(i * 5) % 3 for i in range(n)], kv_dtype=kv, seed=48))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_decode_keeps_a_bad_query_to_its_row(api, kv, value):
    wl = W.make_workload("nan", 16, [700, 90, 9000], [2, 1, 1], kv_dtype=kv, seed=49)
    d = Dev(api, wl)
    d.q[1, 3, 5] = value          # no-RoPE part of one head's query; a RoPE value of another's
    d.q[3, 7, 150] = value
    out, lse = d.decode()
    bad = torch.zeros((4, 16), dtype=torch.bool)
    bad[1, 3] = bad[3, 7] = True
    assert bool(torch.isnan(out[bad.cuda()]).any(-1).all()), "a bad query's row is not NaN"
    keep = ~bad.numpy()
    ref = decode_ref(wl)
    o, x = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o[keep]).all()
    assert np.linalg.norm(o[keep] - ref[0][keep]) <= REL_RMS * np.linalg.norm(ref[0][keep])
    assert (np.abs(x[keep] - ref[1][keep]) <= ref[2][keep]).all()


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("where", [0, 511, 515])      # latent values, a RoPE value
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_decode_keeps_a_bad_new_token_from_the_queries_before_it(api, kv, where, value):
    # the last token but one of each request's new ones, in the first tile, behind whole ones, at a tile's start and
    # among many queries: only its own query and the last one see it
    new = [4, 3, 2, 150]
    wl = W.make_workload("nt", 16, [20, 1000, 127, 90], new, kv_dtype=kv, seed=53)
    codes = W.BF16_NAN if value == "nan" else 0xFF80
    rows = np.zeros(sum(new), dtype=bool)
    for r, n in enumerate(wl.seq_lens):
        t = int(n) - 2
        row = wl.kv_cache[wl.block_table[r][t // 64], t % 64]
        if kv == "bf16":
            row[where] = codes
        elif where < 512:
            row[where] = W.E4M3_NAN                    # (E4M3 has no infinity)
        else:
            row[512:].view(np.uint16)[where - 512] = codes
        rows[int(wl.cu_q[r + 1]) - 2:int(wl.cu_q[r + 1])] = True
    out, lse = Dev(api, wl).decode()
    assert api.device_error(api.decode.last_workspace) == 0
    with np.errstate(all="ignore"):
        ref = decode_ref(wl)
    nan = value == "nan" or (kv != "bf16" and where < 512)
    if nan:
        assert bool(torch.isnan(out[torch.from_numpy(rows).cuda()]).all())
    for x in ref[:2]:
        x[rows] = np.nan                               # left out of the comparison
    assert_decode(out, lse, ref)


@gpu
def test_decode_cu_q_that_does_not_ascend_is_reported(api):
    wl = W.make_workload("mix", 16, [300, 90, 1000], [2, 1, 2], seed=54)
    d = Dev(api, wl)
    for cu in ([0, 3, 2, 5], [0, 2, 3, -1], [5, 0, 5, 2]):
        out, lse = d.decode(cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert api.device_error(api.decode.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    out, lse = d.decode()
    assert api.device_error(api.decode.last_workspace) == 0
    assert_decode(out, lse, decode_ref(wl))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_sink_does_not_drown_the_others(api, kv):
    """One key takes about 0.9 of every row's weight, 6000 others share the rest: each of their weights is about
    2^-16 of the largest, and what they add together is there."""
    wl = W.make_workload("sink", 16, [6000], [1], kv_dtype=kv, seed=51)
    rng = np.random.Generator(np.random.PCG64(52))
    wl.q[...] = 0
    wl.q_pos[...] = 0
    qr = W.f32_to_bf16_bits(rng.standard_normal(64, dtype=np.float32))
    wl.q[..., 128:] = qr                                          # every head asks for the same k_rope
    v = bf16_values(qr)
    want = math.log(0.9 / 0.1 * 6000) / wl.softmax_scale          # the sink's score over the others' mean
    sink = W.f32_to_bf16_bits((v / (v @ v) * want).astype(np.float32))
    rows = wl.block_table[0][np.arange(6001) // 64], np.arange(6001) % 64
    b, t = rows[0][77], rows[1][77]
    wl.kv_cache[b, t, 512:] = sink if kv == "bf16" else sink.view(np.uint8)
    # the others' latents share a direction, which stands out of their sum
    c, _ = cache_values(wl.kv_cache[rows], kv, wl.kv_scale)
    c = c * 0.7 + 1.0
    c[77] = 0.125
    if kv == "bf16":
        wl.kv_cache[rows[0], rows[1], :512] = W.f32_to_bf16_bits(c.astype(np.float32))
    else:
        codes = torch.from_numpy((c / wl.kv_scale).clip(-448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
        wl.kv_cache[rows[0], rows[1], :512] = codes.view(torch.uint8).numpy()
    d, out, lse = check_decode(api, wl)
    # the sink alone would give 0.125 of the columns' sums: a good part of the output is the others'
    ref = decode_ref(wl)[0]
    alone = 0.125 * bf16_values(wl.kv_b_proj)[:, 16 * 128:].reshape(512, 16, 128).sum(0)
    assert np.linalg.norm(ref - alone) > 0.3 * np.linalg.norm(ref)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_leaves_rows_behind_the_batch(api, dtype):
    wl = W.make_workload("b", 16, [70, 90, 40], [2, 1, 3], seed=37)
    d = Dev(api, wl)
    out = torch.full((6, 16, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((6, 16), 7.0, device="cuda")
    cu = torch.tensor([0, 2, 3, 3], dtype=torch.int32, device="cuda")
    d.decode(cu_q=cu, out=out, lse=lse)
    assert bool((out[3:] == 7).all()) and bool((lse[3:] == 7).all())
    assert_decode(out, lse, decode_ref(wl, cu=cu.cpu().numpy()))


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("where", [0, 2, 4])
def test_decode_bad_block_reads_zeros(api, kv, where):
    wl = W.make_workload("bb", 16, [300, 200], [1, 1], kv_dtype=kv, seed=38)
    d = Dev(api, wl)
    good, good_lse = d.decode()
    for bad in (-1, wl.num_blocks, -2 ** 31, 2 ** 31 - 1):
        d.block_table[0, where] = bad
        out, lse = d.decode()
        assert api.device_error(api.decode.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
        assert api.device_error(api.decode.last_workspace) == 0      # read and cleared
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        assert_decode(out[1:], lse[1:], tuple(x[1:] for x in decode_ref(wl)))
    zeroed = wl.kv_cache.copy()
    zeroed[wl.block_table[0, where]] = 0
    import dataclasses
    assert_decode(out, lse, decode_ref(dataclasses.replace(wl, kv_cache=zeroed)))


@gpu
def test_decode_sequence_longer_than_its_table(api):
    wl = W.make_workload("lt", 16, [128 - 1], [1], seed=39)
    d = Dev(api, wl)
    d.seq_lens += 1000       # the table holds 128 tokens: the row sees those
    out, lse = d.decode()
    assert api.device_error(api.decode.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    assert_decode(out, lse, decode_ref(wl))


@gpu
def test_decode_repeats_bit_for_bit(api):
    wl = W.make_workload("rep", 64, [5000, 333, 2048], [1, 2, 1], seed=40)
    d = Dev(api, wl)
    a = d.decode()
    ws = api.decode.last_workspace
    ws.fill_(0xAB)           # nothing depends on what a workspace held
    b = d.decode(workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_decode_matches_prefill(api):
    wl = W.make_workload("dp", 128, [2100, 1500], [1, 4], seed=41)
    d = Dev(api, wl)
    out, lse = d.decode()
    ref, ref_lse = api.prefill(d.q, d.q_pos, d.kv_cache, d.block_table, wl.seq_lens, wl.cu_q, d.kv_b_proj,
                               chunk=1024, softmax_scale=wl.softmax_scale, absorbed=True)
    rel = float((out - ref).norm() / ref.norm())
    assert rel <= 2 * REL_RMS                       # each within REL_RMS of the exact values
    assert float((lse - ref_lse).abs().max()) <= 2 * decode_ref(wl)[2].max()


@gpu
def test_decode_blocks_far_into_a_large_pool(api):
    # block offsets past 2^32 bytes, and a block shared by two requests
    nb = (1 << 32) // (64 * 1152) + 50
    wl = W.make_workload("far", 16, [150, 100], [1, 1], seed=42)
    d = Dev(api, wl)
    cache = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    at = nb - wl.num_blocks
    cache[at:] = d.kv_cache
    d.kv_cache, d.block_table = cache, torch.where(d.block_table >= 0, d.block_table + at, d.block_table)
    out, lse = d.decode()
    assert_decode(out, lse, decode_ref(wl))
    d.block_table[1, 0] = d.block_table[0, 0]
    wl.block_table[1, 0] = wl.block_table[0, 0]
    out, lse = d.decode()
    assert_decode(out, lse, decode_ref(wl))


@gpu
def test_decode_refusals(api):
    wl = W.make_workload("ref", 16, [70, 90], [1, 1], seed=43)
    d = Dev(api, wl)
    a = dict(q=d.q, q_pos=d.q_pos, kv_cache=d.kv_cache, block_table=d.block_table, seq_lens=d.seq_lens,
             kv_b_proj=d.kv_b_proj, softmax_scale=0.07)
    seg, ptr = seg_tensors([[], []])
    for kw in (dict(q=d.q.float()), dict(q=d.q.cpu()), dict(q=d.q[:, :, :190]), dict(q=d.q.transpose(0, 1)),
               dict(q_pos=d.q_pos.long()), dict(q_pos=d.q_pos[:1]), dict(kv_cache=d.kv_cache[:, :, :512]),
               dict(block_table=d.block_table[:1]), dict(seq_lens=wl.seq_lens), dict(seq_lens=d.seq_lens.cpu()),
               dict(kv_b_proj=d.kv_b_proj[:, :256]), dict(kv_b_proj=d.kv_b_proj.float()), dict(segments=seg),
               dict(seg_ptr=ptr), dict(segments=seg.int(), seg_ptr=ptr), dict(segments=seg, seg_ptr=ptr[:2]),
               dict(cu_q=ptr[:2]), dict(cu_q=ptr.long()), dict(out=torch.empty((2, 16, 64), device="cuda")),
               dict(out=torch.empty((2, 16, 128), dtype=torch.float16, device="cuda")),
               dict(lse=torch.empty((2, 15), device="cuda")),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(softmax_scale=float("nan")), dict(rope_theta=1.0), dict(q=d.q[:1].expand(3, 16, 192).contiguous(),
                                                                            q_pos=d.q_pos[:1].expand(3).contiguous())):
        with pytest.raises((ValueError, AttributeError, _lib.MLAError)):
            api.decode(**{**a, **kw})
    out = api.decode(d.q[:0], d.q_pos[:0], d.kv_cache, d.block_table, d.seq_lens, d.kv_b_proj, softmax_scale=0.07)
    assert out.shape == (0, 16, 128)


# ------------------------------------------------------------------ as they are used

def step_inputs(wl, steps, seed):
    """Per step: the batch's new cache rows (before norm and rotation) and queries."""
    rng = np.random.Generator(np.random.PCG64(seed))
    B, H = wl.num_reqs, wl.num_heads
    kv = W.f32_to_bf16_bits(2.0 * rng.standard_normal((steps, B, 576), dtype=np.float32))
    q = W.f32_to_bf16_bits(rng.standard_normal((steps, B, H, 192), dtype=np.float32))
    return kv, q


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_loop_in_a_replayed_graph(api, kv):
    """Append and decode captured once and replayed while the sequences grow over a block's end: each step equals
    the eager calls' bit for bit, and the 64-bit values."""
    steps, H = 6, 16
    room = W.make_workload("loop", H, [63 + steps, 200 + steps, 500 + steps], [1, 1, 1], kv_dtype=kv, seed=44)
    lens0 = np.asarray([61, 197, 500], dtype=np.int32)      # 61 .. 67: over a block's end
    new, qs = step_inputs(room, steps, 45)
    weight = W.f32_to_bf16_bits(np.ones(512, dtype=np.float32))
    as_bf16 = lambda x: torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    d = Dev(api, room)
    eager = Dev(api, room)
    kv_in, q_in, lens, pos = as_bf16(new[0]), as_bf16(qs[0]), torch.from_numpy(lens0).cuda(), torch.from_numpy(lens0).cuda()
    w = as_bf16(weight)
    ws = torch.empty(api.decode_workspace_size(3, 3, H), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((3, H, 128), device="cuda"), torch.empty((3, H), device="cuda")

    def step(dd, out, lse, ws):
        api.cache_append(kv_in, pos, dd.kv_cache, dd.block_table, lens, norm_weight=w, kv_scale=room.kv_scale)
        api.decode(q_in, pos, dd.kv_cache, dd.block_table, lens, dd.kv_b_proj, softmax_scale=room.softmax_scale,
                   kv_scale=room.kv_scale, out=out, lse=lse, workspace=ws)

    lens.fill_(1)
    pos.zero_()
    spare = Dev(api, room)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(spare, out, lse, ws)                            # first use outside the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(d, out, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    import dataclasses
    for i in range(steps):
        kv_in.copy_(as_bf16(new[i]))
        q_in.copy_(as_bf16(qs[i]))
        lens.copy_(torch.from_numpy(lens0 + i + 1))
        pos.copy_(torch.from_numpy(lens0 + i))
        graph.replay()
        eo, el = torch.empty_like(out), torch.empty_like(lse)
        step(eager, eo, el, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(out, eo) and torch.equal(lse, el)
        assert torch.equal(d.kv_cache.view(torch.uint8), eager.kv_cache.view(torch.uint8))
        if i in (0, 3, steps - 1):
            cache = d.kv_cache.cpu()
            cache = cache.view(torch.int16).numpy().view(np.uint16) if kv == "bf16" else cache.numpy()
            now = dataclasses.replace(room, kv_cache=cache, q=qs[i], q_pos=(lens0 + i).astype(np.int32),
                                      ctx_lens=lens0 + i, ext_lens=np.ones(3, dtype=np.int32))
            assert_decode(out, lse, decode_ref(now))


@gpu
def test_decode_after_append_equals_prefill_of_the_same_tokens(api):
    """A prompt appended and prefilled, then one token appended and decoded: the decoded row is the last row of
    prefilling all of it."""
    n, H = 1300, 16
    wl = W.make_workload("pd", H, [0], [n], seed=46)
    d = Dev(api, wl)
    rng = np.random.Generator(np.random.PCG64(47))
    kv = torch.from_numpy(W.f32_to_bf16_bits(rng.standard_normal((n, 576), dtype=np.float32)).view(np.int16)).cuda().view(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    api.cache_append(kv[:n - 1], pos[:n - 1], d.kv_cache, d.block_table, lens)
    api.cache_append(kv[n - 1:], pos[n - 1:], d.kv_cache, d.block_table, lens + 1)
    out, lse = api.decode(d.q[n - 1:], pos[n - 1:], d.kv_cache, d.block_table, lens + 1, d.kv_b_proj,
                          softmax_scale=wl.softmax_scale, return_lse=True)
    ref, ref_lse = api.prefill(d.q, pos, d.kv_cache, d.block_table, [n], [0, n], d.kv_b_proj, chunk=1024,
                               softmax_scale=wl.softmax_scale)
    assert float((out - ref[n - 1:]).norm() / ref[n - 1:].norm()) <= 2 * REL_RMS
    assert float((lse - ref_lse[n - 1:]).abs().max()) <= 2e-2     # two 1e-2 lse bounds of 1300 unit-size logits


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_graphs_that_share_a_workspace(api, kv):
    """Two captured calls of different batches on one workspace, first full of other bytes, replayed in turn: each
    replay has its own results, bit for bit."""
    wls = [W.make_workload("g0", 16, [900, 40, 300], [1, 2, 1], kv_dtype=kv, seed=60),
           W.make_workload("g1", 48, [64, 2100], [3, 1], kv_dtype=kv, seed=61)]
    devs = [Dev(api, w) for w in wls]
    want = [d.decode() for d in devs]
    n = max(api.decode_workspace_size(w.num_reqs, w.q.shape[0], w.num_heads) for w in wls)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(o), torch.empty_like(x)) for o, x in want]
    graphs = []
    for d, (o, x) in zip(devs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.decode(out=o, lse=x, workspace=ws)
        graphs.append(g)
    ws.fill_(255)
    for i in (0, 1, 0, 0, 1, 1, 0, 1):
        for o, x in outs:
            o.zero_()
            x.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert api.device_error(ws) == 0
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
        assert not outs[1 - i][0].any()


@gpu
def test_serving_calls_on_two_streams(api):
    """Calls in flight at once on two streams, each with its own workspace, keep to themselves."""
    wls = [W.make_workload("s%d" % i, 64, [3000 + 500 * i, 40], [1, 2], seed=50 + i) for i in range(2)]
    devs = [Dev(api, w) for w in wls]
    want = [d.decode() for d in devs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(api.decode_workspace_size(2, 3, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [(torch.empty_like(o), torch.empty_like(x)) for o, x in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s, w, (o, x) in zip(devs, streams, spaces, outs):
            d.decode(out=o, lse=x, workspace=w, stream=s)
    torch.cuda.synchronize()
    for (o, x), (eo, ex) in zip(outs, want):
        assert torch.equal(o, eo) and torch.equal(x, ex)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_sees_inputs_that_copies_changed_between_calls(api, kv):
    """Calls one behind the other with nothing but copies between them that put other queries, positions, lengths,
    row counts and segments at the same addresses: each call has its own, bit for bit."""
    wl = W.make_workload("cp", 16, [700, 300, 2000], [3, 2, 1], kv_dtype=kv, seed=56)
    d = Dev(api, wl, [[(0, 100, 0)], [(0, 50, 3)], []])
    rng = np.random.Generator(np.random.PCG64(57))
    versions = []
    for cu, lens, segs in (([0, 3, 5, 6], [703, 302, 2001], [(0, 100, 0), (0, 50, 3)]),
                           ([0, 1, 2, 6], [200, 9, 1500], [(10, 30, 5), (0, 5, 1)]),
                           ([0, 0, 6, 6], [40, 290, 1000], [(0, 9, 9), (100, 100, 100)]),
                           ([1, 2, 3, 4], [64, 0, 1999], [(3, 4, 5), (6, 7, 8)])):
        q = W.f32_to_bf16_bits(rng.standard_normal(wl.q.shape, dtype=np.float32))
        x = [torch.from_numpy(q.view(np.int16)).view(torch.bfloat16), torch.from_numpy(rng.integers(0, 10 ** 5, 6, dtype=np.int32)),
             torch.tensor(lens, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), torch.tensor(segs, dtype=torch.int64)]
        versions.append([t.pin_memory() for t in x])
    at = [d.q, d.q_pos, d.seq_lens, d.cu_q, d.segments]
    want = []
    for v in versions:
        own = [t.cuda() for t in v]
        d.q, d.q_pos, d.seq_lens, d.cu_q, d.segments = own
        want.append(d.decode(out=torch.zeros((6, 16, 128), device="cuda"), lse=torch.zeros((6, 16), device="cuda")))
        torch.cuda.synchronize()
    d.q, d.q_pos, d.seq_lens, d.cu_q, d.segments = at
    ws = torch.empty(api.decode_workspace_size(3, 6, 16), dtype=torch.uint8, device="cuda")
    got = [(torch.zeros((6, 16, 128), device="cuda"), torch.zeros((6, 16), device="cuda")) for _ in range(24)]
    torch.cuda.synchronize()
    for i, (o, x) in enumerate(got):
        for t, v in zip(at, versions[i % 4]):
            t.copy_(v, non_blocking=True)
        d.decode(out=o, lse=x, workspace=ws)
    torch.cuda.synchronize()
    assert api.device_error(ws) == 0
    for i, (o, x) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(x, want[i % 4][1]), i


@gpu
def test_decode_allocates_on_the_stream_that_it_runs_on(api):
    """Outputs and workspaces that the call makes itself are not handed to later work of another stream while it runs."""
    wl = W.make_workload("st", 64, [6000, 40], [1, 2], seed=55)
    d = Dev(api, wl)
    want = d.decode()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, junk = [], []
    for _ in range(8):
        got.append(d.decode(stream=side))
        junk.append(torch.full((api.decode_workspace_size(2, 3, 64),), 255, dtype=torch.uint8, device="cuda"))
        del junk[:-1]
    torch.cuda.synchronize()
    for o, x in got:
        assert torch.equal(o, want[0]) and torch.equal(x, want[1])


# ------------------------------------------------------------------ values at the range's ends

def rope_scores(wl, logits, heads):
    """Makes the score of key t of the batch's only request, for head h, logits[t] * heads[h]: no latent query, one
    q_rope at position 0, keys along it (each with its bf16 roundings, as decode_ref has them)."""
    rng = np.random.Generator(np.random.PCG64(70))
    n = int(wl.seq_lens[0])
    qr = rng.standard_normal(64)
    wl.q[...] = 0
    wl.q_pos[...] = 0
    wl.q[..., 128:] = W.f32_to_bf16_bits((np.asarray(heads)[None, :, None] * qr).astype(np.float32))
    t = np.arange(n)
    k = W.f32_to_bf16_bits((np.asarray(logits)[:, None] / wl.softmax_scale * qr / (qr @ qr)).astype(np.float32))
    wl.kv_cache[wl.block_table[0][t // 64], t % 64, 512:] = k if wl.kv_dtype == "bf16" else k.view(np.uint8)


def set_latents(wl, c):
    """Latents of the batch's only request."""
    t = np.arange(c.shape[0])
    if wl.kv_dtype == "bf16":
        x = W.f32_to_bf16_bits(c.astype(np.float32))
    else:
        x = torch.from_numpy((c / wl.kv_scale).clip(-448, 448).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    wl.kv_cache[wl.block_table[0][t // 64], t % 64, :512] = x


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("logit", [1e2, 1e3, 1e4, 1e5])
def test_decode_large_logits(api, kv, sign, logit):
    """The largest logits are logit (1 + h / 16) for head h, of either sign, shared by five equal keys in both halves
    of several tiles; every other key lies at least an eighth of that below, e^-12 and less.  The output is the five
    keys' mean, whatever the error that a score of this size has (2^-9 of it, alike for equal keys)."""
    n, H = 900, 16
    wl = W.make_workload("ll", H, [n - 1], [1], kv_dtype=kv, seed=62)
    rng = np.random.Generator(np.random.PCG64(63))
    x = rng.uniform(-1, 0.875, n) if sign > 0 else rng.uniform(-2, -1.125, n)
    x[[3, 77, 300, 777, 895]] = sign
    rope_scores(wl, logit * x, 1 + np.arange(H) / 16)
    check_decode(api, wl)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("tail", ["equal", "spread"])
@pytest.mark.parametrize("nats", [5, 7, 9, 11, 12, 14])
def test_decode_small_weights_beside_a_sink(api, kv, tail, nats):
    """One key whose latent is 0 lies nats .. nats + 1 above 4095 others, whose latents have no common part: the
    output is made of their weights alone, each e^-nats of the largest.  A weight may be off by 2^-7 of it (the sum
    of two 8-bit terms of three bits each), of standard deviation 2^-7 / sqrt(3) at most, beside the four other
    roundings; the sink's score by nats u / sqrt(3) times sqrt(3 / 64) for 64 products of a normal q_rope with
    itself: sqrt(4 (u / sqrt(3))^2 + (2^-7 / sqrt(3))^2 + (14 u / 8)^2) = 9.4e-3 of the output, below REL_RMS."""
    n, H, B = 4096, 16, 80
    wl = W.make_workload("sw", H, [n - 1], [1], kv_dtype=kv, seed=64)
    rng = np.random.Generator(np.random.PCG64(65))
    x = np.zeros(n) if tail == "equal" else 0.5 * rng.standard_normal(n)
    x[50] = nats
    rope_scores(wl, x, 1 + np.arange(H) / (16 * nats))
    c = rng.standard_normal((n, 512))
    c[50] = 0
    set_latents(wl, c)
    ref = decode_ref(wl)
    # 80 requests over the same rows: each cluster has a whole one's tiles, so that the others stand beside the sink
    d = Dev(api, wl)
    d.q, d.q_pos, d.seq_lens = d.q.repeat(B, 1, 1), d.q_pos.repeat(B), d.seq_lens.repeat(B)
    d.block_table = d.block_table.repeat(B, 1)
    out, lse = d.decode(cu_q=None)
    assert api.device_error(api.decode.last_workspace) == 0
    assert_decode(out, lse, tuple(np.repeat(x, B, 0) for x in ref))


# ------------------------------------------------------------------ caches of another shape

def other_pools(device):
    """Caches of another block size, of flat rows and of another row, of 40 blocks' rows each."""
    shapes = [(160, 16), (20, 128), (2560,), (1, 40, 64), (40, 64, 1)]
    rows = [(torch.bfloat16, 576), (torch.uint8, 640)]
    pools = [torch.zeros(s + (n,), dtype=t, device=device) for s in shapes for t, n in rows]
    return pools + [torch.zeros((40, 64, n), dtype=t, device=device) for t, n in ((torch.bfloat16, 640), (torch.uint8, 576), (torch.float16, 576))]


def test_cache_shapes_are_checked():
    from mla_prefix_cache_gb300 import api as A
    assert A.kv_dtype_code(torch.zeros((3, 64, 576), dtype=torch.bfloat16)) == _lib.KV_BF16
    assert A.kv_dtype_code(torch.zeros((3, 64, 640), dtype=torch.uint8)) == _lib.KV_FP8_E4M3
    for pool in other_pools("cpu"):
        with pytest.raises(ValueError):
            A.kv_dtype_code(pool)


@gpu
def test_calls_refuse_caches_of_another_shape(api):
    wl = W.make_workload("sh", 16, [70, 90], [1, 1], seed=69)
    d = Dev(api, wl)
    kv, ids = torch.ones((2, 576), dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for pool in other_pools("cuda"):
        d.kv_cache = pool
        for call in (lambda: d.decode(),
                     lambda: api.cache_append(kv, d.q_pos, pool, d.block_table, d.seq_lens),
                     lambda: api.gather_latent(pool, d.block_table[0], 0, 1),
                     lambda: api.block_hash(pool, ids),
                     lambda: api.block_compare(pool, ids, ids),
                     lambda: api.prefill(d.q, d.q_pos, pool, d.block_table, wl.seq_lens, wl.cu_q, d.kv_b_proj, chunk=128,
                                         softmax_scale=wl.softmax_scale)):
            with pytest.raises(ValueError):
                call()
        assert not pool.view(torch.uint8).any()


@gpu
@pytest.mark.parametrize("n", [0, -1, -5, -2 ** 31 + 5, -2 ** 31 + 1, -2 ** 31])
def test_append_leaves_requests_of_negative_length_out(api, n):
    c = append_case([70, 66, 80], [3, 5, 4], "bf16", seed=10)
    c["lens"][1] = n
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_append(c, run_append(api, c, dev_error=err))
    assert int(err.item()) == 0


@gpu
@pytest.mark.parametrize("kv, where", [("bf16", 3), ("bf16", 515), ("fp8_e4m3", 515)])    # a latent value, a RoPE value
@pytest.mark.parametrize("token", [5, 200, 515, 598])    # in an inner tile, in the last one, a new one but the last
@pytest.mark.parametrize("H", [16, 64])                  # 64 rows of an item of 128, two whole items
def test_decode_infinite_key(api, kv, where, token, H):
    """An infinite latent makes a query that sees it NaN whatever its score's sign, an infinite k_rope where the
    score is +infinite; at -infinite it leaves nothing of the key.  The tile's place changes nothing."""
    wl = W.make_workload("inf", H, [596], [4], kv_dtype=kv, seed=68)
    rot = turn(bf16_values(wl.q)[..., 128:], angles(wl.q_pos.astype(np.int64))[:, None])
    lat = np.einsum("ihd,chd->ihc", bf16_values(wl.q)[..., :128], bf16_values(wl.kv_b_proj)[:, :H * 128].reshape(512, H, 128))
    tol = decode_ref(wl)[2]
    row = wl.kv_cache[wl.block_table[0][token // 64], token % 64]
    if kv == "bf16":
        row[where] = 0x7F80                                                      # +inf
    else:
        row[512:].view(np.uint16)[where - 512] = 0x7F80
    out, lse = Dev(api, wl).decode()
    assert api.device_error(api.decode.last_workspace) == 0
    with np.errstate(all="ignore"):
        ref = decode_ref(wl)
    up = (lat[..., where] if where < 512 else rot[..., where - 512]) > 0     # the score's sign
    sees = token <= 596 + np.arange(4)
    nan = sees[:, None] & (up | (where < 512))
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got).all(-1), nan) and np.array_equal(np.isnan(got).any(-1), nan)
    assert up[sees].any() and not up[sees].all()
    down = sees[:, None] & ~up                                                   # lse without the key
    x = lse.double().cpu().numpy()
    assert np.isnan(x[sees[:, None] & up]).all()
    assert (np.abs(x[down] - ref[1][down]) <= tol[down]).all()
    keep = ~nan
    assert np.linalg.norm(got[keep] - ref[0][keep]) <= REL_RMS * np.linalg.norm(ref[0][keep])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_segments_at_the_ends_of_64_bits(api, kv):
    lo, hi = -2 ** 63, 2 ** 63 - 1
    wl = W.make_workload("s64", 16, [300, 300, 300, 300, 300], [1, 1, 2, 1, 1], kv_dtype=kv, seed=66)
    segs = [[(lo, 1, 0), (10, 20, 5)], [(lo, hi, 0), (0, 7, 0)], [(-5, 10, 3), (hi, 1, 0)], [(hi, hi, 0)],
            [(lo + 1, hi, 0), (2, hi, 9)]]
    check_decode(api, wl, segs)


@gpu
def test_decode_of_no_rows_reports_no_error(api):
    wl = W.make_workload("nr", 16, [70, 90], [1, 1], seed=67)
    d = Dev(api, wl)
    junk = torch.full((api.decode_workspace_size(2, 0, 16),), 255, dtype=torch.uint8, device="cuda")
    del junk                 # the allocator hands its memory to the call
    api.decode(d.q[:0], d.q_pos[:0], d.kv_cache, d.block_table, d.seq_lens, d.kv_b_proj, softmax_scale=0.07)
    assert api.device_error(api.decode.last_workspace) == 0


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("lens, rows, cluster", [
    ([300], 1, 2),                    # 3 tiles and 2 units before them, a cluster each: the first tile's
    ([700] * 40, 2, 0),               # 320 units: the first cluster has an item's first two tiles
    ([0, 5000, 60, 1500], 9, 20),     # 124 units: units 32 and 33, inside the second request
], ids=["one", "pieces", "mixed"])
def test_decode_wait_runs_out_and_reports_timeout(api, monkeypatch, kv, lens, rows, cluster):
    """Failure detection without a fault: one cluster's loads of Q and of the scores' keys are withheld (a test hook of
    the library), so that the waits for them and for all that comes of them run out after the shortened limit.  The
    kernel records MLA_ERR_TIMEOUT, frees its tensor memory and returns, the other clusters' rows are right, and so is
    the next call on the same workspace."""
    wl = W.make_workload("to", 16, lens, [rows] * len(lens), kv_dtype=kv, seed=71)
    d = Dev(api, wl)
    ws = torch.empty(api.decode_workspace_size(len(lens), rows * len(lens), 16), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MLA_WAIT_LIMIT_US", "2000")
    monkeypatch.setenv("MLA_TEST_WITHHOLD_CLUSTER", str(cluster))
    out, lse = d.decode(workspace=ws)
    torch.cuda.synchronize()
    assert api.device_error(ws) == 6                 # MLA_ERR_TIMEOUT
    assert api.device_error(ws) == 0                 # cleared by the read
    monkeypatch.delenv("MLA_TEST_WITHHOLD_CLUSTER")
    monkeypatch.delenv("MLA_WAIT_LIMIT_US")
    ref = decode_ref(wl)
    if len(lens) > 1:                                # the cluster has none of the last request's keys
        last = slice(-rows, None)
        assert_decode(out[last], lse[last], tuple(x[last] for x in ref))
    out, lse = d.decode(workspace=ws)
    assert api.device_error(ws) == 0
    assert_decode(out, lse, ref)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_decode_long_context(api, kv):
    # 131072 tokens, two queries: 2048 blocks, each of 64 distinct ones 32 times in the table
    wl = W.make_workload("lc", 8, [4094], [2], kv_dtype=kv, seed=72)
    wl.block_table = np.tile(wl.block_table[:, :64], (1, 32))
    wl.ctx_lens = wl.ctx_lens + np.int32(31 * 4096)
    wl.q_pos = wl.q_pos + np.int32(31 * 4096)
    check_decode(api, wl)
