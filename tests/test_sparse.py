"""The operators of a sparse decoding step (block tables and slot maps, means of
filled blocks, scores of blocks, the choice of blocks) against plain
implementations in 64 bits, and a run of them with appending and decoding.

Tolerances.  u(t) = torch.finfo(t).eps / 2 is the relative rounding of type t.
 - Tables, slots, chosen blocks and lengths are whole numbers: equal.
 - A mean is an fp32 sum of 64 values and one rounding to bf16: within u(bf16) of
   itself, and within 64 u(fp32) of the mean magnitude of its terms (their sum's
   roundings; E4M3 codes and kv_scale are multiplied in fp32 too).
 - (What block_scores keeps of a score between its two kernels is f16, less the maximum
   of 32 blocks: off by 2^-11 |s - maximum| at most; e_h has that of the widest pair.)
 - A score s_hj = scale (qlat . c_j + qrot . k_j) has operands rounded to bf16 (qlat
   and qrot; the means are given): 576 terms, each off by an independent relative
   error of at most u, standard deviation u / sqrt(3) at most: six of them are
   e_hj = 6 scale u / sqrt(3) sqrt(sum (qlat c_j)^2 + (qrot k_j)^2), plus 2^-15 for the
   fp32 sums, the rotation and the exponentials.  With e_h the largest of a head's,
   every e^{s_hj} is off by a factor of at most e^{e_h} and their sum too, so a share
   is within e^{2 e_h} - 1 of itself, and the mean over the heads within the mean of
   share_hj (e^{2 e_h} - 1); u(out) on top.
"""
import ctypes
import math

import numpy as np
import pytest

from mla_prefix_cache_gb300 import _lib, workload as W
from test_serving import U_BF16, angles, append_case, assert_decode, bf16_values, cache_values, turn

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
U_FP32 = torch.finfo(torch.float32).eps / 2


@pytest.fixture(scope="module")
def api():
    from mla_prefix_cache_gb300 import api as A
    _lib.load()
    return A


@pytest.fixture(scope="module")
def lib():
    from mla_prefix_cache_gb300 import build
    import os
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ references

class Tables:
    """Block tables as lists, by the rules one block at a time."""

    def __init__(self, B, width, pool, seed=0, extra=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.table = np.full((B, width), -1, dtype=np.int32)
        self.held = np.zeros(B, dtype=np.int32)
        self.stack = np.concatenate([rng.permutation(pool), np.full(extra, -7)]).astype(np.int32)
        self.count = pool

    def assign(self, lens, cu=None, shared=None, rows=0):
        """(slots, error bits)."""
        B, width = self.table.shape
        err = 0
        need = []
        for n in lens:
            n = max(int(n), 0)
            err |= 1 if n > 64 * width else 0
            need.append(min(-(-n // 64), width))
        back = []
        for r in range(B):
            keep = min(int(shared[r]), int(self.held[r])) if shared is not None else 0
            for j in range(need[r], int(self.held[r])):
                if j >= keep:
                    back.append(self.table[r, j])
                self.table[r, j] = -1
        for b in reversed(back):
            self.stack[self.count] = b
            self.count += 1
        total, top = 0, self.count
        for r in range(B):
            more = max(0, need[r] - int(self.held[r]))
            total += more
            if total > top:
                err |= 4 if more else 0
                need[r] = min(need[r], int(self.held[r])) if more else need[r]
                continue
            for j in range(int(self.held[r]), need[r]):
                self.count -= 1
                self.table[r, j] = self.stack[self.count]
        self.held[:] = need
        slots = np.full(rows, -1, dtype=np.int64)
        if rows:
            cu = np.arange(B + 1) * (rows // B) if cu is None else cu
            for r in range(B):
                for x in range(max(0, int(cu[r])), min(rows, int(cu[r + 1]))):
                    t = max(int(lens[r]), 0) - (int(cu[r + 1]) - x)
                    if t >= 0 and t // 64 < self.held[r]:
                        slots[x] = int(self.table[r, t // 64]) * 64 + t % 64
        return slots, err


class DevTables:
    def __init__(self, t):
        self.table, self.held, self.stack, self.count = (torch.from_numpy(np.array(x, dtype=np.int32)).cuda()
                                                         for x in (t.table, t.held, t.stack, [t.count]))

    def assign(self, api, lens, cu=None, shared=None, rows=0, **kw):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots = torch.full((rows,), -99, dtype=torch.int64, device="cuda") if rows else None
        api.assign_blocks(self.table, self.held, i32(lens), self.stack, self.count, cu_q=None if cu is None else i32(cu),
                          shared=None if shared is None else i32(shared), slots=slots, dev_error=err, **kw)
        return (np.zeros(0, dtype=np.int64) if slots is None else slots.cpu().numpy()), int(err.item())

    def equals(self, t):
        assert np.array_equal(self.held.cpu().numpy(), t.held)
        assert int(self.count.item()) == t.count
        assert np.array_equal(self.table.cpu().numpy(), t.table)
        assert np.array_equal(self.stack.cpu().numpy(), t.stack)


def scores_ref(q, q_pos, means, table, lens, cu, w, scale, theta=10000.0):
    """(scores, their tolerance without the output's rounding), NaN in rows that no request has."""
    T, H = q.shape[0], q.shape[1]
    out, tol = np.full((T, table.shape[1]), np.nan), np.zeros((T, table.shape[1]))
    wk = w[:, :H * 128].reshape(512, H, 128)
    for r, n in enumerate(lens):
        n = min(max(int(n), 0), 64 * table.shape[1])
        for x in range(int(cu[r]), int(cu[r + 1])):
            t = n - (int(cu[r + 1]) - x)
            out[x] = -np.inf
            b = max(t, 0) // 64
            if b == 0:
                continue
            m = means[table[r, :b]]
            lat = np.einsum("hd,chd->hc", q[x, :, :128], wk)
            rot = turn(q[x, :, 128:], angles(int(q_pos[x]), theta))
            s = scale * (lat @ m[:, :512].T + rot @ m[:, 512:].T)
            e = (6 * scale * U_BF16 / math.sqrt(3) * np.sqrt((lat ** 2) @ (m[:, :512] ** 2).T + (rot ** 2) @ (m[:, 512:] ** 2).T)).max(1) + 2.0 ** -15 + 2.0 ** -11 * np.ptp(s, axis=1)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[x, :b] = p.mean(0)
            tol[x, :b] = (p * np.expm1(2 * e)[:, None]).mean(0)
    return out, tol


def select_ref(scores, table, lens, cu, keep, sinks, recent):
    T = scores.shape[0]
    out, n_out = np.full((T, keep), -1, dtype=np.int32), np.zeros(T, dtype=np.int32)
    for r, n in enumerate(lens):
        n = min(max(int(n), 0), 64 * table.shape[1])
        for x in range(max(0, int(cu[r])), min(T, int(cu[r + 1]))):
            t = n - (int(cu[r + 1]) - x)
            if t < 0:
                continue
            b = t // 64 + 1
            if b <= keep:
                chosen = list(range(b))
            else:
                rest = range(sinks, b - recent)
                best = sorted(rest, key=lambda j: (math.isnan(scores[x, j]), -scores[x, j] if not math.isnan(scores[x, j]) else 0.0, j))
                chosen = sorted(list(range(sinks)) + best[:keep - sinks - recent] + list(range(b - recent, b)))
            out[x, :len(chosen)] = table[r, chosen]
            n_out[x] = 64 * (len(chosen) - 1) + t % 64 + 1
    return out, n_out


def paged(lens, rng, spare=3, width=None):
    need = [-(-max(int(n), 0) // 64) for n in lens]
    pool = sum(need) + spare
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), width or max(need + [1])), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, pool


# ------------------------------------------------------------------ host checks

def test_assign_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)

    def call(bt=d, mb=4, held=d, sl=d, sh=None, B=2, free=d, cap=8, count=d, cu=None, rows=4, slots=d):
        return lib.mla_assign_blocks(bt, mb, held, sl, sh, B, free, cap, count, cu, rows, slots, None, None)
    for b in (dict(bt=None), dict(mb=0), dict(mb=1 << 26), dict(held=None), dict(sl=None), dict(B=0), dict(B=-1), dict(free=None),
              dict(cap=-1), dict(count=None), dict(rows=5), dict(rows=-1), dict(slots=None)):
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(B=8193, rows=0) == _lib.MLA_ERR_UNSUPPORTED
    assert call(B=4096, mb=1 << 19, rows=0) == _lib.MLA_ERR_UNSUPPORTED
    assert call(cap=2 ** 31 - 1) == _lib.MLA_ERR_UNSUPPORTED
    assert call(B=0, rows=0, bt=None) == _lib.MLA_OK


def test_means_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)

    def call(cache=d, kvt=0, scale=1.0, nb=8, bt=d, mb=4, sl=d, cu=d, B=2, rows=5, means=d):
        return lib.mla_block_means(cache, kvt, scale, nb, bt, mb, sl, cu, B, rows, means, None, None)
    for b in (dict(cache=None), dict(cache=ctypes.c_void_p(4104)), dict(kvt=2), dict(nb=0), dict(bt=None), dict(mb=0), dict(sl=None),
              dict(cu=None), dict(B=0), dict(B=-1), dict(rows=-1), dict(means=None), dict(means=ctypes.c_void_p(4104)),
              dict(kvt=1, scale=0.0), dict(kvt=1, scale=float("nan"))):
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(rows=0, cache=None) == _lib.MLA_OK


def test_scores_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)
    n = lib.mla_block_scores_workspace_size(5, 8, 300)
    assert n >= 256 + 5 * 8 * (1152 + 300 * 2 + 10 * 8)
    for T, H, mb in ((5, 0, 4), (5, 129, 4), (-1, 8, 4), (5, 8, 0), (5, 8, 1 << 26), (65536, 1, 4)):
        assert lib.mla_block_scores_workspace_size(T, H, mb) == 0

    def call(q=d, pos=d, means=d, nb=8, bt=d, mb=300, sl=d, cu=d, B=2, T=5, H=8, w=d, sm=0.07, theta=1e4, out=d, od=0, ws=d, wb=n):
        return lib.mla_block_scores(q, pos, means, nb, bt, mb, sl, cu, B, T, H, w, sm, theta, out, od, ws, wb, None)
    for b in (dict(q=None), dict(q=ctypes.c_void_p(4104)), dict(pos=None), dict(means=None), dict(means=ctypes.c_void_p(4104)), dict(nb=0),
              dict(bt=None), dict(mb=0), dict(sl=None), dict(cu=None), dict(B=0), dict(B=-2), dict(T=-1), dict(H=0), dict(w=None),
              dict(w=ctypes.c_void_p(4098)), dict(sm=0.0), dict(sm=float("nan")), dict(theta=0.5), dict(out=None), dict(od=2),
              dict(out=ctypes.c_void_p(4104))):
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(H=129) == call(T=65536) == _lib.MLA_ERR_UNSUPPORTED
    for b in (dict(ws=None), dict(ws=ctypes.c_void_p(4104)), dict(wb=n - 1)):
        assert call(**b) == _lib.MLA_ERR_WORKSPACE, b
    assert call(T=0, q=None) == _lib.MLA_OK


def test_select_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)

    def call(sc=d, dt=0, bt=d, mb=4, sl=d, cu=d, B=2, T=5, keep=8, sinks=1, recent=2, table=d, lens=d):
        return lib.mla_select_blocks(sc, dt, bt, mb, sl, cu, B, T, keep, sinks, recent, table, lens, None, None)
    for b in (dict(sc=None), dict(dt=2), dict(bt=None), dict(mb=0), dict(sl=None), dict(cu=None), dict(B=0), dict(T=-1), dict(keep=0),
              dict(sinks=-1), dict(recent=0), dict(recent=9), dict(sinks=7), dict(sinks=2 ** 31 - 1), dict(table=None), dict(lens=None)):
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(keep=1 << 26) == _lib.MLA_ERR_UNSUPPORTED
    assert call(T=0, sc=None) == _lib.MLA_OK


def test_sparse_validates_without_gpu(lib):
    d = ctypes.c_void_p(4096)
    n = lib.mla_decode_sparse_workspace_size(2, 5, 8, 300, 16)
    assert n >= lib.mla_block_scores_workspace_size(5, 8, 300) + lib.mla_decode_workspace_size(5, 5, 8) + 5 * (300 + 16 + 2) * 4
    for B, T, H, mb, k in ((-1, 5, 8, 4, 4), (2, -1, 8, 4, 4), (2, 5, 129, 4, 4), (2, 5, 0, 4, 4), (2, 5, 8, 0, 4), (2, 5, 8, 4, 0), (2, 5, 8, 4, 1 << 25)):
        assert lib.mla_decode_sparse_workspace_size(B, T, H, mb, k) == 0

    def call(q=d, pos=d, cache=d, kvt=0, scale=1.0, nb=8, means=d, bt=d, mb=300, sl=d, cu=d, B=2, T=5, H=8, keep=16, sinks=1, recent=2, w=d,
             sm=0.07, theta=1e4, out=d, od=0, ws=d, wb=n):
        return lib.mla_decode_sparse(q, pos, cache, kvt, scale, nb, means, bt, mb, sl, cu, B, T, H, keep, sinks, recent, w, sm, theta, out, od,
                                     None, ws, wb, None)
    for b in (dict(q=None), dict(q=ctypes.c_void_p(4104)), dict(pos=None), dict(cache=None), dict(kvt=2), dict(nb=0), dict(means=None),
              dict(means=ctypes.c_void_p(4104)), dict(bt=None), dict(mb=0), dict(sl=None), dict(cu=None), dict(B=0), dict(T=-1), dict(H=0),
              dict(keep=0), dict(sinks=-1), dict(recent=0), dict(sinks=15), dict(w=None), dict(sm=0.0), dict(theta=1.0), dict(out=None), dict(od=2),
              dict(kvt=1, scale=0.0)):
        assert call(**b) == _lib.MLA_ERR_INVALID_ARG, b
    assert call(H=129) == call(T=65536) == call(keep=1 << 26) == call(nb=1 << 25) == call(kvt=1, scale=2.0 ** 33) == _lib.MLA_ERR_UNSUPPORTED
    for b in (dict(ws=None), dict(ws=ctypes.c_void_p(4104)), dict(wb=n - 1)):
        assert call(**b) == _lib.MLA_ERR_WORKSPACE, b
    assert call(T=0, q=None) == _lib.MLA_OK


def test_sparse_keep_beyond_the_table_without_gpu(lib):
    """More kept blocks than a table has ask for no more room and refuse no more work than as many as it has."""
    size = lib.mla_decode_sparse_workspace_size
    most = (2 ** 31 - 1) // 64
    for T, H, mb in ((5, 8, 300), (300, 128, 1), (4000, 16, 2000)):
        assert size(2, T, H, mb, most) == size(2, T, H, mb, mb + 1) == size(2, T, H, mb, mb) > 0
    d = ctypes.c_void_p(4096)

    def call(T, keep, wb):      # sizes are taken up to the workspace's
        return lib.mla_decode_sparse(d, d, d, 0, 1.0, 8, d, d, 300, d, d, 2, T, 128, keep, 1, 2, d, 0.07, 1e4, d, 0, None, d, wb, None)
    for keep in (300, 301, most):
        assert call(4000, keep, size(2, 4000, 128, 300, 300) - 1) == _lib.MLA_ERR_WORKSPACE


def test_documented_limits_without_gpu(lib):
    """The sizes that mla.h names as the first that a call refuses, and the last before them (which then miss a workspace)."""
    d, most = ctypes.c_void_p(4096), 2 ** 25 - 1
    taken, refused = _lib.MLA_ERR_WORKSPACE, _lib.MLA_ERR_UNSUPPORTED

    def scores(T, B, mb):
        return lib.mla_block_scores(d, d, d, 8, d, mb, d, d, B, T, 8, d, 0.07, 1e4, d, 0, None, 0, None)
    assert scores(2048, 2047, most) == taken and scores(2048, 2048, most) == refused          # 2^12 rows and requests, 2^19 tiles
    assert scores(65535, 2 ** 25 - 65536, 64 * 64) == taken and scores(65535, 2 ** 25 - 65535, 64 * 64) == refused
    assert scores(65535, 1, 64) == taken and scores(65536, 1, 64) == refused

    def sparse(T, keep, mb, H=128, nb=8):
        return lib.mla_decode_sparse(d, d, d, 0, 1.0, nb, d, d, mb, d, d, 1, T, H, keep, 1, 2, d, 0.07, 1e4, d, 0, None, None, 0, None)
    # 2 * 2048 * (k / 2 + 5) reaches 2^31 at k = 2^20 - 10
    assert sparse(2048, 2 ** 20 - 11, 2 ** 21) == taken and sparse(2048, 2 ** 20 - 10, 2 ** 21) == refused
    assert sparse(2048, most, 2 ** 20 - 11) == taken and sparse(2048, most, 2 ** 20 - 10) == refused
    assert sparse(1, most, 64) == taken and sparse(1, most + 1, 64) == refused
    assert sparse(1, 4, 64, nb=most) == taken and sparse(1, 4, 64, nb=most + 1) == refused
    assert lib.mla_select_blocks(d, 0, d, 64, d, d, 1, 1, most + 1, 1, 2, d, d, None, None) == refused

    def assign(B, mb, cap, rows=0):
        return lib.mla_assign_blocks(d, mb, d, d, None, B, d, cap, d, d, rows, d, None, None)
    assert assign(8193, 1, 1) == refused and assign(64, most, 64) == refused
    assert assign(32, 2 ** 25 - 1, 2 ** 30 - 2 ** 20 + 32) == refused and assign(1, 1, 1, rows=2 ** 31 - 2 ** 20) == refused


WIDE = [2 ** 32 + 5, 2 ** 31, -2 ** 31 - 1, 5 - 2 ** 32]      # that the library's ints would cut to 5, and to the other sign


@pytest.mark.parametrize("n", WIDE)
def test_numbers_beyond_32_bits_are_refused_without_gpu(lib, n):
    """A count that does not fit the library's ints is an error, not another count.  (It is looked at before the tensors, which are not there.)"""
    from mla_prefix_cache_gb300 import api
    some = dict(block_table=None, seq_lens=None)
    for kw in (dict(keep=n), dict(keep=8, sinks=n), dict(keep=8, recent=n)):
        with pytest.raises(_lib.MLAError):
            api.select_blocks(None, **some, **kw)
        with pytest.raises(_lib.MLAError):
            api.decode_sparse(None, None, None, None, **some, kv_b_proj=None, softmax_scale=0.07, **kw)
    with pytest.raises(_lib.MLAError):
        api.block_means(None, **some, means=None, rows=n)
    with pytest.raises(_lib.MLAError):
        api.decode_sparse_workspace_size(1, 1, 16, 4, n)


def test_reference_tables_undo_themselves():
    t = Tables(3, 6, 12)
    t.assign([65, 0, 200])
    before = (t.table.copy(), t.stack.copy(), t.count)
    slots, err = t.assign([65 + 70, 1, 200 + 60], cu=[0, 70, 71, 131], rows=131)
    assert err == 0 and slots.min() >= 0 and len(set(slots)) == 131
    t.assign([65, 0, 200])
    assert np.array_equal(t.table, before[0]) and np.array_equal(t.stack, before[1]) and t.count == before[2]


# ------------------------------------------------------------------ block tables

STEPS = {
    "one": (1, [[1], [64], [65], [0]]),
    "drafts": (40, [list(range(100, 900, 20)), list(range(104, 904, 20)), list(range(101, 901, 20))]),
    "mixed": (7, [[700, 0, 64, 1, 65, 128, 3], [0, 640, 64, 130, 0, 127, 3], [-5, 640, 63, 129, 64, 0, -2 ** 31]]),
    "many": (1100, [[(7 * r) % 300 for r in range(1100)], [(11 * r + 5) % 300 for r in range(1100)], [0] * 1100]),
    "most": (8192, [[64 * (r % 3) for r in range(8192)], [64 * ((r + 1) % 3) for r in range(8192)]]),
    "wide": (2, [[131072, 1], [1, 131072], [70000, 60000]]),
}


@gpu
@pytest.mark.parametrize("shared", [False, True], ids=["own", "shared"])
@pytest.mark.parametrize("name", STEPS)
def test_assign_matches_the_rules(api, name, shared):
    B, steps = STEPS[name]
    sh = None
    width = max(-(-max(n, 0) // 64) for s in steps for n in s) + 2
    pool = max(sum(-(-max(n, 0) // 64) for n in s) for s in steps) + 3
    t = Tables(B, width, pool, seed=len(name))
    d = DevTables(t)
    for k, lens in enumerate(steps):
        if shared and k:      # leading blocks of what is held that are not the request's own
            sh = [int(h) // 2 + (r % 2) for r, h in enumerate(t.held)]
        new = [min(max(n, 0), (5 * r + k) % 90) for r, n in enumerate(lens)]
        cu = np.cumsum([0] + new)
        a, b = t.assign(lens, cu, sh, rows=int(cu[-1])), d.assign(api, lens, cu, sh, rows=int(cu[-1]))
        assert a[1] == b[1]
        assert np.array_equal(a[0], b[0])
        d.equals(t)


@gpu
def test_assign_uniform_rows_and_rows_of_no_request(api):
    t = Tables(3, 5, 20)
    d = DevTables(t)
    a, b = t.assign([5, 70, 1], rows=6), d.assign(api, [5, 70, 1], rows=6)
    assert np.array_equal(a[0], b[0]) and b[0][4] == -1      # (the one token's first row has a negative token)
    cu = [2, 4, 4, 9]
    a, b = t.assign([5, 70, 100], cu, rows=12), d.assign(api, [5, 70, 100], cu, rows=12)
    assert np.array_equal(a[0], b[0]) and (b[0][:2] == -1).all() and (b[0][9:] == -1).all()
    d.equals(t)


@gpu
@pytest.mark.parametrize("pool", [0, 1, 3, 5, 6])
def test_assign_runs_out(api, pool):
    """Requests are served in order while their blocks are there; what one gives back serves another in the same call."""
    t = Tables(5, 4, pool)
    d = DevTables(t)
    for lens in ([64, 129, 0, 200, 1], [0, 129, 64, 200, 1], [0, 0, 0, 0, 256], [300, 300, 300, 300, 300]):
        cu = np.cumsum([0] + [min(n, 3) for n in lens])
        a, b = t.assign(lens, cu, rows=int(cu[-1])), d.assign(api, lens, cu, rows=int(cu[-1]))
        assert a[1] == b[1]
        assert np.array_equal(a[0], b[0])
        d.equals(t)


@gpu
def test_assign_reports_bad_state(api):
    t = Tables(2, 4, 6, extra=2)
    d = DevTables(t)
    d.held[0] = 9                                   # more than the table is wide: cut to it
    assert d.assign(api, [256, 64])[1] == 1
    assert d.held.tolist() == [4, 1]
    d.count[0] = -3
    assert d.assign(api, [256, 128])[1] == 1 | 4    # no block left, and a count that cannot be
    assert d.held.tolist() == [4, 1] and d.count.item() == 0
    d.count[0] = 8                                  # the stack is full: the entry behind it is lost
    guard = d.stack.clone()
    assert d.assign(api, [256, 0])[1] == 1
    assert torch.equal(d.stack, guard) and d.held.tolist() == [4, 0]


class Prefixed:
    """Requests behind a common prefix of `sh` blocks, of which a pool of others is to be whole at any time.  The mirror of shared[] follows the rule
    that a request which grows from fewer blocks than its shared ones owns what it gets."""

    def __init__(self, B, sh, width, pool, seed=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.B, self.sh, self.width, self.pool = B, sh, width, pool
        table = np.full((B, width), -1, dtype=np.int32)
        table[:, :sh] = pool + np.arange(sh)
        self.table, self.held, self.shared = i32(table), i32([sh] * B), i32([sh] * B)
        self.stack, self.count, self.lens = i32(rng.permutation(pool)), i32([pool]), i32([64 * sh] * B)
        self.err, self.slots = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((2 * B,), -9, dtype=torch.int64, device="cuda")
        self.mirror = np.full(B, sh)

    def call(self, api):
        api.assign_blocks(self.table, self.held, self.lens, self.stack, self.count, shared=self.shared, slots=self.slots, dev_error=self.err)

    def step(self, lens, call):
        before = self.held.cpu().numpy()
        self.lens.copy_(i32(lens))
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        table, held, count, slots = self.table.cpu().numpy(), self.held.cpu().numpy(), int(self.count.item()), self.slots.cpu().numpy()
        stack = self.stack.cpu().numpy()[:count]
        mine = table[(table >= 0) & (table < self.pool)]
        assert np.array_equal(np.sort(np.concatenate([stack, mine])), np.arange(self.pool)), "a block is lost or there twice"
        self.mirror = np.where((held > before) & (self.mirror > before), before, self.mirror)
        assert np.array_equal(self.shared.cpu().numpy(), self.mirror)
        for r in range(self.B):
            assert (table[r, :held[r]] >= 0).all() and (table[r, held[r]:] == -1).all()
            for i in range(2):
                t = lens[r] - 2 + i
                assert slots[2 * r + i] == (table[r, t // 64] * 64 + t % 64 if 0 <= t < 64 * held[r] else -1)
        served = [min(-(-n // 64), self.width) == h for n, h in zip(lens, held)]
        assert int(self.err.item()) == (0 if all(served) else 4)
        self.err.zero_()


@gpu
def test_assign_below_a_shared_prefix_loses_no_block(api):
    """Cut below the prefix, grown again and retired, with shared[] left alone: what was popped below the prefix comes back."""
    t = Prefixed(3, 4, 9, 20)
    for lens in ([6 * 64, 5 * 64 - 3, 300], [2 * 64, 0, 4 * 64], [7 * 64, 3 * 64, 1], [0, 0, 0], [64, 512, 9 * 64], [0, 0, 0]):
        t.step(lens, lambda: t.call(api))
    assert t.count.item() == 20 and t.shared.tolist() == [0, 0, 0]


@gpu
@pytest.mark.parametrize("B, pool", [(5, 200), (5, 24), (40, 150), (1500, 9000)])
def test_assign_below_a_shared_prefix_in_a_replayed_graph(api, B, pool):
    """The same over random lengths, one captured call replayed, with requests put behind the prefix again and a pool that runs out."""
    t = Prefixed(B, 3, 12, pool, seed=B)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        t.call(api)                    # nothing changes hands
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            t.call(api)

    def replay():
        with torch.cuda.stream(stream):
            graph.replay()
    rng = np.random.Generator(np.random.PCG64(pool))
    for k in range(25):
        t.step([int(n) for n in np.where(rng.random(B) < 0.3, 0, rng.integers(0, 64 * 12 + 1, B))], replay)
        if k % 5 == 4:                 # everyone ends, half of them begin again behind the prefix
            t.step([0] * B, replay)
            t.table[::2, :3] = i32(pool + np.arange(3))
            t.held[::2] = 3
            t.shared[::2] = 3
            t.mirror[::2] = 3
    t.step([0] * B, replay)
    assert t.count.item() == pool


@gpu
def test_assign_refusals(api):
    t = Tables(2, 4, 6)
    d = DevTables(t)
    lens = i32([1, 2])
    ok = dict(block_table=d.table, held=d.held, seq_lens=lens, free_blocks=d.stack, free_count=d.count)
    bad = [dict(block_table=d.table.cpu()), dict(block_table=d.table[:1]), dict(block_table=d.table.long()), dict(block_table=d.table.t()),
           dict(held=d.held[:1]), dict(held=d.held.long()), dict(seq_lens=lens.cpu()), dict(free_blocks=d.stack.long()),
           dict(free_blocks=d.stack[::2]), dict(free_blocks=d.stack[None]), dict(free_count=d.stack[:2]), dict(shared=lens.long()), dict(shared=lens[:1]),
           dict(slots=torch.zeros(4, dtype=torch.int32, device="cuda")), dict(slots=torch.zeros(3, dtype=torch.int64, device="cuda")),
           dict(slots=torch.zeros(4, dtype=torch.int64)), dict(cu_q=i32([0, 1]), slots=torch.zeros(1, dtype=torch.int64, device="cuda")),
           dict(dev_error=torch.zeros(1, device="cuda"))]
    for b in bad:
        with pytest.raises(ValueError):
            api.assign_blocks(**{**ok, **b})
    api.assign_blocks(**ok)


# ------------------------------------------------------------------ means

def means_case(lens, new, kv_dtype, seed=0, extra_rows=0):
    c = append_case(lens, new, kv_dtype, seed=seed, extra_rows=extra_rows)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    if kv_dtype == "bf16":
        c["cache"] = W.f32_to_bf16_bits(rng.standard_normal(c["cache"].shape[:2] + (576,), dtype=np.float32)).view(np.uint8)
    else:
        codes = rng.integers(0, 0x7F, c["cache"].shape[:2] + (512,), dtype=np.uint8) | (rng.integers(0, 2, c["cache"].shape[:2] + (512,), dtype=np.uint8) << 7)
        c["cache"] = np.concatenate([codes, W.f32_to_bf16_bits(rng.standard_normal(c["cache"].shape[:2] + (64,), dtype=np.float32)).view(np.uint8)], -1)
    c["means"] = W.f32_to_bf16_bits(rng.standard_normal((c["cache"].shape[0], 576), dtype=np.float32))
    return c


def run_means(api, c, rows=None, uniform=False, cu=None, **kw):
    cache = torch.from_numpy(c["cache"].copy()).cuda()
    if c["kv_dtype"] == "bf16":
        cache = cache.view(torch.bfloat16)
    means = torch.from_numpy(c["means"].view(np.int16).copy()).cuda().view(torch.bfloat16)
    got = api.block_means(cache, torch.from_numpy(c["table"]).cuda(), i32(c["lens"]), means, rows=int(c["cu"][-1]) if rows is None else rows,
                          cu_q=None if uniform else i32(c["cu"] if cu is None else cu), kv_scale=c["scale"], **kw)
    assert got is means
    return bf16_values(means.view(torch.int16).cpu().numpy().view(np.uint16))


def check_means(c, got, cu=None, left=()):
    cu = c["cu"] if cu is None else cu
    before = bf16_values(c["means"])
    rows = c["cache"].view(np.uint16) if c["kv_dtype"] == "bf16" else c["cache"]
    filled = 0
    for r, n in enumerate(c["lens"]):
        k = int(cu[r + 1] - cu[r])
        for j in range(max(int(n) - k, 0) // 64, max(int(n), 0) // 64):
            if (r, j) in left:
                continue
            b = int(c["table"][r, j])
            v = np.concatenate(cache_values(rows[b], c["kv_dtype"], c["scale"]), -1)
            want, size = v.mean(0), np.abs(v).mean(0)
            assert (np.abs(got[b] - want) <= U_BF16 * np.abs(want) + 64 * U_FP32 * size).all(), (r, j)
            before[b] = got[b]
            filled += 1
    assert np.array_equal(got, before), "another row of the means changed"
    return filled


MEANS = {
    "one": ([64], [1]),
    "none": ([63, 65, 1, 127], [1, 1, 1, 62]),                      # no block is filled
    "ragged": ([130, 64, 65, 1, 700, 128], [3, 64, 65, 1, 257, 128]),
    "step": ([64 * (r % 5) + (r % 3) for r in range(1, 201)], [1 + (r % 4 if r > 4 else 0) for r in range(1, 201)]),
    "empty": ([90, 0, 128, 64], [2, 0, 0, 64]),
    "long": ([2000, 5000], [1999, 3333]),
    # more candidates than two an SM
    "ring": ([9000, 7003, 64, 5000], [9000, 6900, 1, 5000]),
    "ring_requests": ([60 + 3 * (r % 50) for r in range(700)], [1 + r % 7 for r in range(700)]),
    "ring_none": ([64 * 5 + 40] * 400, [7] * 400),
}


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("name", MEANS)
def test_means_match_64_bits(api, name, kv):
    lens, new = MEANS[name]
    new = [min(n, k) for n, k in zip(lens, new)]
    c = means_case(lens, new, kv, seed=len(name))
    n = check_means(c, run_means(api, c))
    assert (n == 0) == (name in ("none", "ring_none"))


@gpu
@pytest.mark.parametrize("reqs", [1, 31, 33, 1025])
def test_means_uniform_batch(api, reqs):
    lens = [64 + (13 * r) % 130 for r in range(reqs)]
    c = means_case(lens, [4] * reqs, "bf16", seed=reqs)
    check_means(c, run_means(api, c, rows=4 * reqs, uniform=True))


@gpu
def test_means_leaves_padding_and_other_requests_out(api):
    c = means_case([64, 0, 128, 192], [64, 0, 128, 64], "bf16")
    c["lens"][1], c["lens"][2] = -5, 0                              # padded requests
    cu = np.array([3, 67, 67, 67, 131])                             # rows before the first one and behind the last
    check_means(c, run_means(api, c, rows=140, cu=cu), cu=cu)
    c["lens"][3] = 60                                               # fewer tokens than rows
    check_means(c, run_means(api, c, rows=140, cu=cu), cu=cu)


@gpu
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("n", [200, 21000])
def test_means_bad_block_is_reported(api, bad, n):
    c = means_case([n, 130], [n, 130], "bf16")
    c["table"] = c["table"].copy()
    c["table"][0, 1] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_means(c, run_means(api, c, dev_error=err), left={(0, 1)})
    assert err.item() == 1
    c = means_case([n, 130], [n, 130], "bf16")
    rows = max(64, n - 200)
    c["lens"] = np.array([64 * (c["table"].shape[1] + 1), 130], dtype=np.int32)      # longer than its table
    c["cu"] = np.array([0, rows, rows + 130], dtype=np.int32)
    err.zero_()
    check_means(c, run_means(api, c, dev_error=err), left={(0, c["table"].shape[1])})
    assert err.item() == 1


@gpu
@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0])
def test_means_keep_what_is_not_finite_to_itself(api, value):
    c = means_case([128], [128], "bf16")
    b = c["table"][0]
    c["cache"].view(np.uint16)[b[0], 17, 33] = value
    got = run_means(api, c)
    assert not np.isfinite(got[b[0], 33]) and np.isfinite(np.delete(got[b[0]], 33)).all() and np.isfinite(got[b[1]]).all()


@gpu
@pytest.mark.parametrize("kv, blocks", [("bf16", 7), ("bf16", 3), ("bf16", 2), ("fp8_e4m3", 9)])
@pytest.mark.parametrize("cta", [0, 151])
def test_means_wait_runs_out_and_reports_timeout(api, monkeypatch, kv, blocks, cta):
    """Failure detection without a fault: one CTA takes no block out of its ring (a test hook of the library), so that its loads' wait for room runs
    out after the shortened limit.  It records the timeout, waits for the copies in flight and returns; the others' means are right, and so is
    the next call.  (A ring with room left behind all its blocks waits for none, and reports nothing.)"""
    n = 152 * blocks                                  # CTA c has the blocks c, c + 152, ...
    c = means_case([64 * n], [64 * n], kv)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("MLA_WAIT_LIMIT_US", "2000")
    monkeypatch.setenv("MLA_TEST_WITHHOLD_MEANS", str(cta))
    got = run_means(api, c, dev_error=err)
    torch.cuda.synchronize()
    assert err.item() == (2 if blocks >= (3 if kv == "bf16" else 5) else 0)
    monkeypatch.delenv("MLA_TEST_WITHHOLD_MEANS")
    monkeypatch.delenv("MLA_WAIT_LIMIT_US")
    check_means(c, got, left={(0, j) for j in range(cta, n, 152)})
    err.zero_()
    check_means(c, run_means(api, c, dev_error=err))
    assert err.item() == 0


@gpu
def test_means_refusals(api):
    cache = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda")
    means = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    ok = dict(kv_cache=cache, block_table=i32([[0, 1], [2, 3]]), seq_lens=i32([64, 64]), means=means, rows=128)
    for b in (dict(kv_cache=cache.cpu()), dict(kv_cache=cache[:, :32]), dict(kv_cache=cache.float()), dict(means=means.float()), dict(means=means[:3]),
              dict(means=means[:, :512]), dict(means=means.cpu()), dict(rows=127), dict(seq_lens=i32([64])), dict(block_table=i32([0, 1])),
              dict(cu_q=i32([0, 64]))):
        with pytest.raises(ValueError):
            api.block_means(**{**ok, **b})
    with pytest.raises(_lib.MLAError):
        api.block_means(**{**ok, "rows": -2})
    api.block_means(**ok)
    api.block_means(**{**ok, "rows": 0})


# ------------------------------------------------------------------ scores

class Scores:
    """A batch to be scored: queries, means in a paged pool, and its reference."""

    def __init__(self, lens, q, H, seed=0, cu=None, T=None, theta=10000.0, spread=2.5, width=None):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.lens = np.asarray(lens, dtype=np.int32)
        self.cu = np.cumsum([0] + ([q] * len(lens) if isinstance(q, int) else list(q))) if cu is None else np.asarray(cu)
        T = int(self.cu[-1]) if T is None else T
        self.table, pool = paged(lens, rng, width=width)
        bits = lambda x: W.f32_to_bf16_bits(x.astype(np.float32))  # noqa: E731
        self.means, self.q = bits(0.4 * rng.standard_normal((pool, 576))), bits(spread * rng.standard_normal((T, H, 192)))
        self.w = bits(rng.standard_normal((512, H * 256)) / math.sqrt(512))
        self.pos, self.scale, self.theta, self.H = rng.integers(0, 200000, T).astype(np.int32), 192 ** -0.5, theta, H

    def run(self, api, dtype=torch.float32, **kw):
        d = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
        kw.setdefault("cu_q", i32(self.cu))
        out = api.block_scores(d(self.q), i32(self.pos), d(self.means), torch.from_numpy(self.table).cuda(), i32(self.lens), d(self.w),
                               softmax_scale=self.scale, rope_theta=self.theta, out_dtype=dtype, **kw)
        return out

    def ref(self):
        return scores_ref(bf16_values(self.q), self.pos, bf16_values(self.means), self.table, self.lens, self.cu, bf16_values(self.w),
                          self.scale, self.theta)

    def check(self, out, ref=None):
        want, tol = self.ref() if ref is None else ref
        got, u = out.double().cpu().numpy(), torch.finfo(out.dtype).eps / 2
        rows = ~np.isnan(want[:, :1]).all(1) if want.shape[1] else np.ones(len(want), bool)
        got, want, tol = got[rows], want[rows], tol[rows]
        dead = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), dead)
        live = ~dead
        assert np.isfinite(got[live]).all()
        e, most = np.abs(got[live] - want[live]), tol[live] + u * (want[live] + tol[live]) + 2.0 ** -126
        assert (e <= most).all(), f"{(e / most).max():.2f} of the bound"


SCORES = [
    ("first", [1, 63, 64, 65, 128, 129], 1, 16),             # no block, one block
    ("one_tile", [64 * 128 + 1, 64 * 129, 64 * 127 + 5], 1, 128),
    ("ragged", [20000, 64, 9000, 100, 0, 8256], 1, 40),
    ("drafts", [500, 64 * 40 + 2, 8195, 64], 4, 32),         # rows on both sides of a block's border
    ("heads", [3000, 700], 2, 1),
    ("heads_odd", [9000, 64, 2500], 3, 100),
    ("wide", [64 * 600], 5, 7),
    ("ends", [700, 2000, 30], [9, 0, 30], 16),
    ("many", [200 + 37 * r for r in range(150)], 1, 8),
    ("items", [70 + 19 * (r % 97) for r in range(330)], 1, 128),                 # several items of full rows a CTA
    ("items_drafts", [70 + 83 * (r % 41) for r in range(170)], 3, 48),
    ("requests", [(37 * r) % 500 if r % 3 else 0 for r in range(1100)], [1 if r % 3 else 0 for r in range(1100)], 8),      # more than a CTA's threads
    ("few_of_many", [9000 + 64 * (r % 50) if r % 7 == 0 else 0 for r in range(620)], [1 if r % 7 == 0 else 0 for r in range(620)], 16),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", SCORES, ids=[c[0] for c in SCORES])
def test_scores_match_64_bits(api, case, dtype):
    name, lens, q, H = case
    s = Scores(lens, q, H, seed=len(name))
    s.check(s.run(api, dtype))
    assert api.device_error(api.block_scores.last_workspace) == 0


@gpu
def test_scores_uniform_batch_on_a_wide_table(api):
    s = Scores([900, 64, 4000], 2, 16, width=300, theta=500000.0)
    s.check(s.run(api, cu_q=None))


@gpu
@pytest.mark.parametrize("logits", [20, 300, 3000])
def test_scores_peaked(api, logits):
    """One block has nearly all of a head's attention: shares stay shares, however large the scores are."""
    s = Scores([6000, 9000], 1, 16, spread=2.5 * logits / 10)
    out = s.run(api)
    live = ~torch.isinf(out)
    assert torch.isfinite(out[live]).all() and (out[live] >= 0).all()
    total = torch.where(live, out, torch.zeros_like(out)).sum(1)
    # each share is rounded in its exponential and the reference is its own maximum: sums of 1 but for fp32's roundings
    assert (total - 1).abs().max() <= 2.0 ** -13
    if logits == 20:
        s.check(out)


def share_bounds(s, x):
    """(least, largest) share of each block of query x, whatever the scores' size.  s_hj is off by at most e_hj: the operands' roundings as in the file's
    head, 576 fp32 additions of 2^-23 of the terms' magnitude, the f16's 2^-11 of the distance to a maximum, and 2^-15 of that distance (or of 1) for
    the rotation and the exponentials.  A share is largest with its own score up by e and the others' down, least the other way round."""
    r = int(np.searchsorted(s.cu, x, side="right")) - 1
    b = (int(s.lens[r]) - (int(s.cu[r + 1]) - x)) // 64
    q, w, m = bf16_values(s.q)[x], bf16_values(s.w)[:, :s.H * 128].reshape(512, s.H, 128), bf16_values(s.means)[s.table[r, :b]]
    v = np.concatenate([np.einsum("hd,chd->hc", q[:, :128], w), turn(q[:, 128:], angles(int(s.pos[x]), s.theta))], 1)
    z = s.scale * (v @ m.T)
    far = z.max(1, keepdims=True) - z
    e = s.scale * (6 * U_BF16 / math.sqrt(3) * np.sqrt((v ** 2) @ (m ** 2).T) + 576 * 2.0 ** -23 * (np.abs(v) @ np.abs(m).T))
    e = e + 2.0 ** -11 * (far + e + e.max(1, keepdims=True)) + 2.0 ** -15 * np.maximum(1, far)

    def share(mine, others):
        d = others[:, None, :] - mine[:, :, None]
        i = np.arange(b)
        d[:, i, i] = 0.0
        with np.errstate(over="ignore"):      # (infinitely less)
            return (1 / np.exp(d).sum(2)).mean(0)
    return share(z - e, z + e), share(z + e, z - e)


def peaked(logits):
    return Scores([6000, 9000, 64 * 70 + 1], 1, 16, spread=2.5 * logits / 10, seed=logits)


@pytest.mark.parametrize("logits", [300, 3000])
def test_share_bounds_tell_blocks_apart(logits):
    """The bounds hold for the reference itself, and not for its shares moved to the next block."""
    s = peaked(logits)
    want = s.ref()[0]
    for x in range(3):
        lo, hi = share_bounds(s, x)
        p = want[x, :len(lo)]
        assert (lo <= p * (1 + 1e-9)).all() and (p <= hi * (1 + 1e-9) + 1e-300).all()
        moved = np.roll(p, 1)
        assert (moved < lo).any() and (moved > hi).any()
        assert lo.sum() > 0.6                 # most heads' largest block is certain


@gpu
@pytest.mark.parametrize("logits", [20, 300, 3000])
def test_scores_peaked_blocks(api, logits):
    """Which blocks have the heads' attention, where scores are far apart and most of what leaves the score kernel is -infinite."""
    s = peaked(logits)
    out = s.run(api).double().cpu().numpy()
    for x in range(3):
        lo, hi = share_bounds(s, x)
        p = out[x, :len(lo)]
        # (the heads' sum and its last rounding: 32 of fp32)
        assert (p >= lo * (1 - 32 * U_FP32) - 2.0 ** -126).all() and (p <= hi * (1 + 32 * U_FP32) + 2.0 ** -126).all()


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", [0, 511, 575])
def test_scores_keep_what_is_not_seen_out(api, value, where):
    """A block that is not finite leaves NaN in the queries that see it, and nothing in the others, of its own request or another one."""
    s = Scores([64 * 130 + 3, 64 * 20], 8, 16)
    want = s.ref()
    bits = W.f32_to_bf16_bits(np.float32([value]))[0]
    s.means = s.means.copy()
    s.means[s.table[0, 129], where] = bits         # the first five rows of request 0 lie in this block, the last three behind it
    s.means[s.table[1, 19], where] = bits
    out = s.run(api)
    assert torch.isnan(out[5:8, :130]).all()
    want[0][5:8] = np.nan
    s.check(out, want)


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_scores_keep_a_bad_query_to_its_row(api, value):
    s = Scores([3000, 5000], 3, 16)
    want = s.ref()
    s.q = s.q.copy()
    s.q[1, 5, 40] = W.f32_to_bf16_bits(np.float32([value]))[0]
    s.q[4, 0, 150] = W.f32_to_bf16_bits(np.float32([value]))[0]
    out = s.run(api)
    for x in (1, 4):
        seen = ~np.isneginf(want[0][x])
        assert torch.isnan(out[x, :int(seen.sum())]).all() and torch.isneginf(out[x, int(seen.sum()):]).all()
        want[0][x] = np.nan
    s.check(out, want)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_leave_rows_of_no_request(api, dtype):
    s = Scores([700, 9000], 2, 16, cu=[2, 4, 6], T=9)
    out = torch.full((9, s.table.shape[1]), 7.0, dtype=dtype, device="cuda")
    s.run(api, out=out)
    assert (out[:2] == 7).all() and (out[6:] == 7).all()
    s.check(out)


@gpu
def test_scores_report_bad_batches(api):
    s = Scores([3000, 9000], 2, 16)
    want = s.ref()
    # a bad block id scores as a mean of zeros
    s.table = s.table.copy()
    good, s.table[1, 7] = s.table[1, 7], 10 ** 6
    out = s.run(api)
    assert api.device_error(api.block_scores.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    s.table[1, 7], s.means = good, s.means.copy()
    s.means[good] = 0
    s.check(out)
    # longer than its table: cut off there
    s.lens[0] = 64 * s.table.shape[1] + 5
    s.table[0] = s.table[1]
    out = s.run(api)
    assert api.device_error(api.block_scores.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    s.check(out)
    # a cu_q that does not ascend: nothing is scored
    out = s.run(api, cu_q=i32([0, 3, 2]))
    assert api.device_error(api.block_scores.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    assert not torch.isfinite(out[:2]).any()
    out = s.run(api)
    s.check(out)


@gpu
def test_scores_refusals(api):
    q = torch.zeros((2, 16, 192), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((512, 16 * 256), dtype=torch.bfloat16, device="cuda")
    means = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, q_pos=i32([5, 6]), means=means, block_table=i32([[0, 1], [2, 3]]), seq_lens=i32([70, 70]), kv_b_proj=w, softmax_scale=0.07)
    bad = [dict(q=q.cpu()), dict(q=q.float()), dict(q=q[..., :128]), dict(q=q[:, ::2]), dict(q_pos=i32([5])), dict(q_pos=torch.zeros(2, device="cuda")),
           dict(means=means.float()), dict(means=means[:, :512]), dict(means=means.cpu()), dict(kv_b_proj=w[:, :256]), dict(block_table=i32([0, 1])),
           dict(seq_lens=i32([70])), dict(cu_q=i32([0, 1])), dict(out=torch.zeros((2, 3), device="cuda")), dict(out=torch.zeros((2, 2), device="cuda").half()),
           dict(out=torch.zeros((2, 2)))]
    for b in bad:
        with pytest.raises(ValueError):
            api.block_scores(**{**ok, **b})
    for b in (dict(softmax_scale=0.0), dict(rope_theta=1.0), dict(workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(_lib.MLAError):
            api.block_scores(**{**ok, **b})
    api.block_scores(**ok)
    out = api.block_scores(**{**ok, "q": q[:0], "q_pos": ok["q_pos"][:0]})
    assert out.shape == (0, 2) and api.device_error(api.block_scores.last_workspace) == 0


# ------------------------------------------------------------------ selection

def select_case(lens, q, seed=0, ties=False, width=None, dtype=torch.float32):
    rng = np.random.Generator(np.random.PCG64(seed))
    cu = np.cumsum([0] + ([q] * len(lens) if isinstance(q, int) else list(q)))
    table, _ = paged(lens, rng, width=width)
    x = rng.standard_normal((int(cu[-1]), table.shape[1]))
    x = rng.integers(-2, 3, x.shape) * 0.25 if ties else np.where(x < -1, 0.0, np.exp(2 * x))
    return torch.tensor(x, dtype=torch.float32).to(dtype), table, np.asarray(lens, dtype=np.int32), cu


def check_select(api, scores, table, lens, cu, keep, sinks, recent, uniform=False, **kw):
    got = api.select_blocks(scores.cuda(), torch.from_numpy(table).cuda(), i32(lens), keep=keep, sinks=sinks, recent=recent,
                            cu_q=None if uniform else i32(cu), **kw)
    want = select_ref(scores.double().numpy(), table, lens, cu, keep, sinks, recent)
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[0].cpu().numpy(), want[0])


SELECT = [
    ([1], 1, 1, 0, 1), ([64, 65, 128, 0, 63], 1, 2, 0, 1), ([5000, 300, 64 * 32, 64 * 32 + 1, 64 * 33], 1, 32, 1, 2),
    ([9000, 700], 8, 16, 3, 3), ([64 * 300 + 5] * 3, 2, 6, 3, 3), ([64 * 9 + 1, 64 * 257 + 1, 64 * 256, 64 * 513], 1, 7, 0, 1),
    ([200000, 150001], 1, 64, 1, 2), ([40000], 4, 500, 4, 100), ([70, 500], [7, 33], 3, 1, 1), ([64 * 700], 1, 699, 0, 1),
    ([300001, 262000], 1, 40, 1, 2), ([64 * 4095, 64 * 100], 1, 33, 1, 2), ([64 * 16383 + 1, 20000], 1, 64, 2, 3), ([64 * 16400 + 7], 2, 64, 1, 2),
    ([700000], 1, 3000, 1, 2), ([250000], 1, 2500, 0, 7),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("ties", [False, True], ids=["spread", "ties"])
@pytest.mark.parametrize("case", SELECT)
def test_select_matches_the_rules(api, case, ties, dtype):
    lens, q, keep, sinks, recent = case
    check_select(api, *select_case(lens, q, len(lens), ties, dtype=dtype), keep, sinks, recent)


@gpu
@pytest.mark.parametrize("keep", [3, 4, 20, 149, 150, 151, 152, 153])
def test_select_every_number_and_a_uniform_batch(api, keep):
    check_select(api, *select_case([64 * 151, 64 * 151 - 60], 2, keep, keep % 2 == 1, width=200), keep, 1, 2, uniform=True)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_select_odd_scores(api, dtype):
    """NaN below everything, infinities at the ends, -0 as 0, subnormal scores apart from 0, all scores alike."""
    scores, table, lens, cu = select_case([64 * 400 + 9] * 4, 1, dtype=dtype)
    scores[0, 5:300:3] = float("nan")
    scores[0, 7:300:5] = float("inf")
    scores[0, 9:390:4] = float("-inf")
    scores[1] = 0.0
    scores[1, ::2] = -0.0
    scores[2] = float("nan")
    scores[3] = 1e-39
    scores[3, 100:200] = 2e-39
    scores[3, 300:310] = -1e-39
    for keep in (5, 40, 250, 399):
        check_select(api, scores, table, lens, cu, keep, 1, 2)


@gpu
def test_select_reads_nothing_that_is_not_seen(api):
    scores, table, lens, cu = select_case([64 * 50 + 1, 64 * 10], 3, width=80)
    want = [x.clone() for x in api.select_blocks(scores.cuda(), torch.from_numpy(table).cuda(), i32(lens), keep=12, cu_q=i32(cu))]
    for x in range(6):
        own = (int(lens[x // 3]) - 3 + x % 3) // 64
        scores[x, own - 1:] = float("inf")
        scores[x, :1] = float("nan")
    got = api.select_blocks(scores.cuda(), torch.from_numpy(table).cuda(), i32(lens), keep=12, cu_q=i32(cu))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_select_rows_of_no_request_and_long_sequences(api):
    scores, table, lens, _ = select_case([700, 300, 64], 2)
    check_select(api, torch.cat([scores, scores]), table, np.array([700, 300, 1]), np.array([2, 4, 6, 8]), 5, 1, 2)     # (a negative token in the last one)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_select(api, scores, table, np.array([64 * table.shape[1] + 100, 300, -3]), np.array([0, 2, 4, 6]), 5, 1, 2, dev_error=err)
    assert err.item() == 1


@gpu
def test_select_refusals(api):
    s, t, n = torch.zeros((2, 8), device="cuda"), i32(np.zeros((2, 8))), i32([500, 500])
    for b in (dict(scores=s.cpu()), dict(scores=s.half()), dict(scores=s[:, :4]), dict(scores=s.t()), dict(scores=s[0]), dict(seq_lens=n[:1]),
              dict(table=i32(np.zeros((2, 3)))), dict(table=torch.zeros((2, 4), dtype=torch.int64, device="cuda")), dict(lens=i32([1])),
              dict(cu_q=i32([0, 2]))):
        with pytest.raises(ValueError):
            api.select_blocks(**{**dict(scores=s, block_table=t, seq_lens=n, keep=4), **b})
    for b in (dict(keep=0), dict(sinks=-1), dict(recent=0), dict(sinks=3)):
        with pytest.raises(_lib.MLAError):
            api.select_blocks(s, t, n, **{**dict(keep=4), **b})
    api.select_blocks(s, t, n, keep=4)


# ------------------------------------------------------------------ the attention, and all of it together

class Topics:
    """A cache whose blocks are about one of some topics, and queries that ask for one: which blocks are chosen does not hang on roundings.

    A topic is a direction of the latents, `about` says which one a block has (-1: none) and `asks` which one a query row asks for."""

    def __init__(self, api, lens, q, H, kv, keep, sinks, recent, seed=0, cu=None, T=None):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.api, self.kv, self.H, self.lens = api, kv, H, np.asarray(lens, dtype=np.int32)
        self.keep, self.sinks, self.recent = keep, sinks, recent
        self.cu = np.cumsum([0] + ([q] * len(lens) if isinstance(q, int) else list(q))) if cu is None else np.asarray(cu)
        T = int(self.cu[-1]) if T is None else T
        self.T = T
        self.table, pool = paged(lens, rng)
        bits = lambda x: W.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))  # noqa: E731
        self.w = bits(rng.standard_normal((512, H * 256)) / math.sqrt(512))
        wk = bf16_values(self.w)[:, :H * 128].reshape(512, H, 128)
        topics = rng.standard_normal((len(lens), 512))
        x = rng.standard_normal((pool, 64, 576)).astype(np.float32)
        for r, n in enumerate(lens):
            first = max(0, n - int(self.cu[r + 1] - self.cu[r])) // 64           # the first query's own block
            free = np.arange(sinks, max(sinks, (first if first + 1 > keep else max(n - 1, 0) // 64) + 1 - recent))
            for j in rng.permutation(free)[:keep - sinks - recent]:
                x[self.table[r, j], :, :512] += topics[r]
        self.q = rng.standard_normal((T, H, 192))
        for r in range(len(lens)):
            self.q[self.cu[r]:self.cu[r + 1], :, :128] += 0.5 * np.einsum("c,chd->hd", topics[r], wk)
        self.q = bits(self.q)
        self.pos = np.zeros(T, dtype=np.int32)
        for r, n in enumerate(lens):
            self.pos[self.cu[r]:self.cu[r + 1]] = np.arange(n - (self.cu[r + 1] - self.cu[r]), n)
        self.scale, self.kv_scale = 192 ** -0.5, 1.0
        if kv == "bf16":
            self.cache = bits(x)
        else:
            self.kv_scale = 6.0 / 448.0
            codes = torch.from_numpy(x[..., :512] / self.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            self.cache = np.concatenate([codes, bits(x[..., 512:]).view(np.uint8)], -1)
        c, k = cache_values(self.cache, kv, self.kv_scale)
        self.means = bits(np.concatenate([c, k], -1).mean(1))

    def dev(self):
        d = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
        cache = d(self.cache) if self.kv == "bf16" else torch.from_numpy(self.cache).cuda()
        return dict(q=d(self.q), q_pos=i32(self.pos), kv_cache=cache, means=d(self.means), block_table=torch.from_numpy(self.table).cuda(),
                    seq_lens=i32(self.lens), kv_b_proj=d(self.w))

    def run(self, dev=None, **kw):
        a = dict(keep=self.keep, sinks=self.sinks, recent=self.recent, softmax_scale=self.scale, kv_scale=self.kv_scale, return_lse=True)
        a.update(kw)
        if "cu_q" not in kw:
            a["cu_q"] = i32(self.cu)
        return self.api.decode_sparse(**(dev or self.dev()), **a)

    def ref(self):
        """(out, lse, lse tolerance) as decode's reference has it, over the blocks that the scores' reference chooses."""
        H = self.H
        shares = scores_ref(bf16_values(self.q), self.pos, bf16_values(self.means), self.table, self.lens, self.cu, bf16_values(self.w), self.scale)[0]
        table, n = select_ref(shares, self.table, self.lens, self.cu, self.keep, self.sinks, self.recent)
        q, w = bf16_values(self.q), bf16_values(self.w)
        wk, wv = w[:, :H * 128].reshape(512, H, 128), w[:, H * 128:].reshape(512, H, 128)
        out, lse, tol = np.full((self.T, H, 128), np.nan), np.full((self.T, H), np.nan), np.zeros((self.T, H))
        for x in range(int(self.cu[0]), int(self.cu[-1])):
            if n[x] == 0:
                out[x], lse[x] = 0.0, -np.inf
                continue
            t = np.arange(n[x])
            c, k = cache_values(self.cache[table[x][t // 64], t % 64], self.kv, self.kv_scale)
            lat = np.einsum("hd,chd->hc", q[x, :, :128], wk)
            rot = turn(q[x, :, 128:], angles(int(self.pos[x])))
            s = self.scale * (lat @ c.T + rot @ k.T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            lse[x] = m[:, 0] + np.log(p.sum(1))
            out[x] = np.einsum("hc,chd->hd", (p / p.sum(1, keepdims=True)) @ c, wv)
            tol[x] = 6 * self.scale * U_BF16 / math.sqrt(3) * np.sqrt(((lat ** 2) @ (c ** 2).T + (rot ** 2) @ (k ** 2).T).max(1)) + 2.0 ** -15
        return out, lse, tol


SPARSE = [
    ("short", [1, 64, 65, 200], 1, 16, 4, 1, 2),                                    # every block chosen
    ("one", [5000], 1, 128, 12, 1, 2),
    ("ragged", [20000, 700, 9000, 64, 0, 130], 1, 40, 16, 1, 1),
    ("drafts", [64 * 30 + 2, 1200, 64 * 12], 4, 32, 8, 0, 1),                       # rows on both sides of a block's border
    ("ends", [3000, 900, 1500], [9, 0, 3], 16, 10, 2, 3),
    ("many", [300 + 53 * r for r in range(60)], 1, 8, 7, 1, 2),
    ("requests", [130 + (29 * r) % 200 for r in range(600)], 1, 4, 3, 1, 1),      # more than a CTA's threads
]


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("width", [4097, 16385])
def test_sparse_on_wide_tables(api, kv, width):
    """The choice's forms for long rows, with the attention's plan beside them."""
    t = Topics(api, [3000, 64 * 40 + 1, 500, 64], 2, 16, kv, 9, 1, 2)
    t.table = np.pad(t.table, ((0, 0), (0, width - t.table.shape[1])), constant_values=-1)
    out, lse = t.run()
    assert_decode(out, lse, t.ref())


@gpu
@pytest.mark.parametrize("lens, cta", [([3000], 0), ([3000, 700], 0)])
def test_scores_wait_runs_out_and_reports_timeout(api, monkeypatch, lens, cta):
    """Failure detection without a fault: one CTA's loads of mean rows are withheld (a test hook of the library), so that the
    waits for them run out after the shortened limit.  The kernel records MLA_ERR_TIMEOUT, frees its tensor memory and
    returns, and the next call on the same workspace is right."""
    s = Scores(lens, 1, 16)
    ws = torch.empty(api.block_scores_workspace_size(len(lens), 16, s.table.shape[1]), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MLA_WAIT_LIMIT_US", "2000")
    monkeypatch.setenv("MLA_TEST_WITHHOLD_SCORES", str(cta))
    out = s.run(api, workspace=ws)
    torch.cuda.synchronize()
    assert api.device_error(ws) == _lib.MLA_ERR_TIMEOUT
    assert api.device_error(ws) == 0                 # cleared by the read
    monkeypatch.delenv("MLA_TEST_WITHHOLD_SCORES")
    monkeypatch.delenv("MLA_WAIT_LIMIT_US")
    if len(lens) > 1:                                # the CTA has none of the last request's blocks
        want, tol = s.ref()
        want[0] = np.nan
        s.check(out, (want, tol))
    out = s.run(api, workspace=ws)
    assert api.device_error(ws) == 0
    s.check(out)


@gpu
@pytest.mark.parametrize("lens, cta, spoiled", [([3000, 700], 1, 1), ([64 * 140, 700], 0, 0), ([64 * 140, 700], 1, 0), ([64 * 140, 700], 2, 0), ([64 * 140, 700], 3, 1)])
def test_scores_wait_runs_out_in_any_cta(api, monkeypatch, lens, cta, spoiled):
    """As above, with the first, a middle and the last tile of a request withheld: the other request's scores are right."""
    s = Scores(lens, 1, 16, seed=cta)
    ws = torch.empty(api.block_scores_workspace_size(2, 16, s.table.shape[1]), dtype=torch.uint8, device="cuda")
    want, tol = s.ref()
    part = want.copy()
    part[spoiled] = np.nan
    monkeypatch.setenv("MLA_WAIT_LIMIT_US", "2000")
    monkeypatch.setenv("MLA_TEST_WITHHOLD_SCORES", str(cta))
    out = s.run(api, workspace=ws)
    torch.cuda.synchronize()
    assert api.device_error(ws) == _lib.MLA_ERR_TIMEOUT
    monkeypatch.delenv("MLA_TEST_WITHHOLD_SCORES")
    monkeypatch.delenv("MLA_WAIT_LIMIT_US")
    s.check(out, (part, tol))
    s.check(s.run(api, workspace=ws), (want, tol))
    assert api.device_error(ws) == 0


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_wait_runs_out_and_reports_timeout(api, monkeypatch, kv):
    """The whole call with one CTA's mean rows withheld: it reports, ends, and the next one on the same workspace is right."""
    t = Topics(api, [3000, 700], 1, 16, kv, 8, 1, 2)
    d = t.dev()
    ws = torch.empty(api.decode_sparse_workspace_size(2, 2, 16, t.table.shape[1], 8), dtype=torch.uint8, device="cuda")
    want = [x.clone() for x in t.run(d, workspace=ws)]
    for cta in (0, 1):
        monkeypatch.setenv("MLA_WAIT_LIMIT_US", "2000")
        monkeypatch.setenv("MLA_TEST_WITHHOLD_SCORES", str(cta))
        t.run(d, workspace=ws)
        torch.cuda.synchronize()
        assert api.device_error(ws) == _lib.MLA_ERR_TIMEOUT
        monkeypatch.delenv("MLA_TEST_WITHHOLD_SCORES")
        monkeypatch.delenv("MLA_WAIT_LIMIT_US")
        out, lse = t.run(d, workspace=ws)
        assert api.device_error(ws) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", SPARSE, ids=[c[0] for c in SPARSE])
def test_sparse_matches_64_bits(api, case, kv):
    name, lens, q, H, keep, sinks, recent = case
    t = Topics(api, lens, q, H, kv, keep, sinks, recent, seed=len(name))
    out, lse = t.run()
    assert api.device_error(api.decode_sparse.last_workspace) == 0
    assert_decode(out, lse, t.ref())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_uniform_batch_bf16_out_without_lse(api, kv):
    t = Topics(api, [3000, 4100, 500], 2, 32, kv, 9, 1, 2)
    out = t.run(cu_q=None, return_lse=False, out_dtype=torch.bfloat16)
    assert out.dtype is torch.bfloat16
    assert_decode(out, None, t.ref())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_is_its_parts(api, kv):
    """Bit for bit what scores, choice and decode give one after another; with every block kept, what decode gives."""
    t = Topics(api, [3000, 64 * 40 + 1, 500, 64], 2, 32, kv, 9, 1, 2)
    d = t.dev()
    out, lse = t.run(d)
    scores = api.block_scores(d["q"], d["q_pos"], d["means"], d["block_table"], d["seq_lens"], d["kv_b_proj"], softmax_scale=t.scale)
    table, lens = api.select_blocks(scores, d["block_table"], d["seq_lens"], keep=t.keep, sinks=t.sinks, recent=t.recent)
    a = dict(softmax_scale=t.scale, kv_scale=t.kv_scale, return_lse=True)
    want = api.decode(d["q"], d["q_pos"], d["kv_cache"], table, lens, d["kv_b_proj"], **a)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out, lse = t.run(d, keep=d["block_table"].shape[1])
    # (a request of one row each, as the sparse form has it: the same cut of the work)
    every = d["block_table"].repeat_interleave(2, 0).contiguous()
    want = api.decode(d["q"], d["q_pos"], d["kv_cache"], every, (d["q_pos"] + 1).contiguous(), d["kv_b_proj"], **a)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("q", [1, 3])
def test_sparse_keeps_every_block_of_a_narrow_table(api, kv, q):
    """A keep above the table's width, with first and recent blocks above it too: bit for bit what the width gives."""
    t = Topics(api, [3000, 64 * 40 + 1, 500, 64], q, 32, kv, 9, 1, 2)
    d = t.dev()
    width = d["block_table"].shape[1]
    ws = torch.empty(api.decode_sparse_workspace_size(4, 4 * q, 32, width, width), dtype=torch.uint8, device="cuda")
    want = [x.clone() for x in t.run(d, keep=width, workspace=ws)]
    for kw in (dict(keep=width + 1), dict(keep=50 * width, sinks=2 * width, recent=3 * width), dict(keep=(2 ** 31 - 1) // 64)):
        out, lse = t.run(d, workspace=ws, **kw)
        assert api.device_error(ws) == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_leaves_rows_of_no_request(api, kv):
    t = Topics(api, [3000, 900], 2, 16, kv, 9, 1, 2, cu=[2, 4, 6], T=9)
    out, lse = torch.full((9, 16, 128), 7.0, device="cuda"), torch.full((9, 16), 7.0, device="cuda")
    t.run(out=out, lse=lse)
    assert (out[:2] == 7).all() and (out[6:] == 7).all() and (lse[:2] == 7).all() and (lse[6:] == 7).all()
    assert_decode(out, lse, t.ref())


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_reports_bad_batches(api, kv):
    t = Topics(api, [3000, 2000], 1, 16, kv, 8, 1, 2)
    d = t.dev()
    good = t.run(d)
    bad = dict(d, block_table=d["block_table"].clone())
    bad["block_table"][0, 3] = 10 ** 6                       # scored as zeros
    t.run(bad)
    assert api.device_error(api.decode_sparse.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    bad["block_table"][0, 3] = d["block_table"][0, 3]
    bad["block_table"][1, 0] = -1                            # and a chosen one, attended as zeros
    t.run(bad)
    assert api.device_error(api.decode_sparse.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    long = dict(d, seq_lens=d["seq_lens"].clone())
    long["seq_lens"][0] = 64 * d["block_table"].shape[1] + 1
    t.run(long)
    assert api.device_error(api.decode_sparse.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    t.run(d, cu_q=i32([0, 2, 1]))
    assert api.device_error(api.decode_sparse.last_workspace) == _lib.MLA_ERR_BAD_BLOCK_ID
    again = t.run(d)
    assert api.device_error(api.decode_sparse.last_workspace) == 0
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@gpu
def test_sparse_refusals(api):
    t = Topics(api, [300, 200], 1, 16, "bf16", 4, 1, 2)
    d = t.dev()
    for b in (dict(q=d["q"].cpu()), dict(q=d["q"].float()), dict(q_pos=d["q_pos"][:1]), dict(kv_cache=d["kv_cache"][:, :32]), dict(means=d["means"][:2]),
              dict(means=d["means"].float()), dict(means=d["means"].cpu()), dict(block_table=d["block_table"][:1]), dict(kv_b_proj=d["kv_b_proj"][:, :256])):
        with pytest.raises(ValueError):
            t.run({**d, **b})
    for b in (dict(keep=0), dict(sinks=3), dict(recent=0), dict(softmax_scale=-1.0), dict(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(_lib.MLAError):
            t.run(d, **b)
    out = api.decode_sparse(**{**d, "q": d["q"][:0], "q_pos": d["q_pos"][:0]}, keep=4, softmax_scale=0.07)
    assert out.shape == (0, 16, 128) and api.device_error(api.decode_sparse.last_workspace) == 0


class Step:
    """A speculative decoding loop over one layer: drafted tokens get blocks, are appended and attended, and are cut back to the accepted ones."""

    def __init__(self, api, kv, B=5, q=3, H=16, keep=6, seed=3):
        rng = np.random.Generator(np.random.PCG64(seed))
        bits = lambda x: torch.from_numpy(W.f32_to_bf16_bits(np.asarray(x, dtype=np.float32)).view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
        self.api, self.kv, self.B, self.q, self.H, self.keep = api, kv, B, q, H, keep
        self.width, pool = 24, 24 * B
        self.w, self.norm = bits(rng.standard_normal((512, H * 256)) / math.sqrt(512)), bits(1 + 0.2 * rng.standard_normal(512))
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.free, self.count = i32(rng.permutation(pool)), i32([pool])
        self.scale = 1.0 if kv == "bf16" else 5.0 / 448
        self.cache = (torch.zeros((pool, 64, 576), dtype=torch.bfloat16, device="cuda") if kv == "bf16"
                      else torch.zeros((pool, 64, 640), dtype=torch.uint8, device="cuda"))
        self.means = torch.zeros((pool, 576), dtype=torch.bfloat16, device="cuda")
        self.rng, self.bits = rng, bits
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, n):
        return self.bits(2 * self.rng.standard_normal((n, 576)))

    def append(self, kv, pos, lens, cu, rows, slots):
        a = self.api
        a.assign_blocks(self.table, self.held, lens, self.free, self.count, cu_q=cu, slots=slots, dev_error=self.err)
        a.cache_append(kv, pos, self.cache, self.table, lens, cu_q=cu, norm_weight=self.norm, kv_scale=self.scale, dev_error=self.err)
        a.block_means(self.cache, self.table, lens, self.means, rows=rows, cu_q=cu, kv_scale=self.scale, dev_error=self.err)

    def prompt(self, lens):
        cu = np.cumsum([0] + list(lens))
        self.lens.copy_(i32(lens))
        self.append(self.rows(int(cu[-1])), i32(np.concatenate([np.arange(n) for n in lens])), self.lens, i32(cu), int(cu[-1]),
                    torch.empty(int(cu[-1]), dtype=torch.int64, device="cuda"))

    def buffers(self):
        T = self.B * self.q
        n = self.api.decode_sparse_workspace_size(self.B, T, self.H, self.width, self.keep)
        return dict(kv=self.rows(T), q=self.bits(self.rng.standard_normal((T, self.H, 192)) * 1.5), accepted=torch.zeros(self.B, dtype=torch.int32, device="cuda"),
                    slots=torch.empty(T, dtype=torch.int64, device="cuda"), out=torch.empty((T, self.H, 128), device="cuda"),
                    lse=torch.empty((T, self.H), device="cuda"), ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def step(self, b):
        """q drafted tokens of each request appended and attended, then cut back to the accepted ones; all of it on the device."""
        lens = self.lens + self.q
        pos = (self.lens[:, None] + torch.arange(self.q, dtype=torch.int32, device="cuda")).reshape(-1).contiguous()
        self.append(b["kv"], pos, lens, None, self.B * self.q, b["slots"])
        self.api.decode_sparse(b["q"], pos, self.cache, self.means, self.table, lens, self.w, keep=self.keep, softmax_scale=192 ** -0.5,
                               kv_scale=self.scale, out=b["out"], lse=b["lse"], workspace=b["ws"])
        self.lens += b["accepted"]
        self.api.assign_blocks(self.table, self.held, self.lens, self.free, self.count, dev_error=self.err)


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_loop_in_a_replayed_graph(api, kv):
    """Twenty speculative steps, captured once and replayed, against the same steps with every length and table on the host."""
    s = Step(api, kv)
    s.prompt([700, 64, 129, 1000, 383])
    b = s.buffers()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        keep = [x.clone() for x in (s.table, s.held, s.free, s.count, s.cache, s.means, s.lens)]
        s.step(b)                                              # a dry run, taken back
        for x, y in zip((s.table, s.held, s.free, s.count, s.cache, s.means, s.lens), keep):
            x.copy_(y)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            s.step(b)
    torch.cuda.synchronize()
    host = Tables(s.B, s.width, 1)
    host.table, host.held, host.stack, host.count = s.table.cpu().numpy(), s.held.cpu().numpy(), s.free.cpu().numpy(), int(s.count.item())
    rng = np.random.Generator(np.random.PCG64(9))
    w = bf16_values(s.w.view(torch.int16).cpu().numpy().view(np.uint16))
    lens = s.lens.cpu().numpy().copy()
    for k in range(20):
        accepted = rng.integers(0, s.q + 1, s.B)
        b["kv"].copy_(s.rows(s.B * s.q))
        b["q"].copy_(s.bits(1.5 * rng.standard_normal((s.B * s.q, s.H, 192))))
        b["accepted"].copy_(i32(accepted))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert s.err.item() == 0 and api.device_error(b["ws"]) == 0
        grown = lens + s.q
        slots, err = host.assign(grown, rows=s.B * s.q)
        assert err == 0 and np.array_equal(slots, b["slots"].cpu().numpy())
        table = host.table.copy()
        # the rows that the graph appended lie in their slots
        rows = s.cache.view(torch.uint8).reshape(-1, s.cache.shape[-1] * s.cache.element_size())[torch.from_numpy(slots).cuda()]
        want = torch.empty_like(s.cache[:1]).repeat(s.B * s.q, 1, 1)
        api.cache_append(b["kv"], i32((lens[:, None] + np.arange(s.q)).reshape(-1)), want, i32(np.arange(s.B * s.q)[:, None]), i32([1] * (s.B * s.q)),
                         norm_weight=s.norm, kv_scale=s.scale)
        assert torch.equal(rows, want.view(torch.uint8).reshape(s.B * s.q, 64, -1)[:, 0])
        if k % 5 == 4:
            cache = s.cache.cpu()
            cache = cache.view(torch.int16).numpy().view(np.uint16) if kv == "bf16" else cache.numpy()
            means = bf16_values(s.means.view(torch.int16).cpu().numpy().view(np.uint16))
            for r in range(s.B):      # every full block's mean, whenever it was filled, and again after a cut
                full = table[r, :grown[r] // 64]
                c = np.concatenate(cache_values(cache[full], kv, s.scale), -1)
                assert (np.abs(means[full] - c.mean(1)) <= U_BF16 * np.abs(c.mean(1)) + 64 * U_FP32 * np.abs(c).mean(1)).all()
            # the attention over the blocks that the device chose
            d = dict(q_pos=i32((lens[:, None] + np.arange(s.q)).reshape(-1)), block_table=torch.from_numpy(table).cuda(), seq_lens=i32(grown))
            sc = api.block_scores(b["q"], d["q_pos"], s.means, d["block_table"], d["seq_lens"], s.w, softmax_scale=192 ** -0.5)
            cu = np.arange(s.B + 1) * s.q
            chosen, n = select_ref(sc.double().cpu().numpy(), table, grown, cu, s.keep, 1, 2)
            qv = bf16_values(b["q"].view(torch.int16).cpu().numpy().view(np.uint16))
            ref = [np.zeros((s.B * s.q, s.H, 128)), np.zeros((s.B * s.q, s.H)), np.zeros((s.B * s.q, s.H))]
            for x in range(s.B * s.q):
                t = np.arange(n[x])
                c, kr = cache_values(cache[chosen[x][t // 64], t % 64], kv, s.scale)
                lat = np.einsum("hd,chd->hc", qv[x, :, :128], w[:, :s.H * 128].reshape(512, s.H, 128))
                rot = turn(qv[x, :, 128:], angles(int(lens[x // s.q]) + x % s.q))
                z = 192 ** -0.5 * (lat @ c.T + rot @ kr.T)
                m = z.max(1, keepdims=True)
                p = np.exp(z - m)
                ref[1][x] = m[:, 0] + np.log(p.sum(1))
                ref[0][x] = np.einsum("hc,chd->hd", (p / p.sum(1, keepdims=True)) @ c, w[:, s.H * 128:].reshape(512, s.H, 128))
                ref[2][x] = 6 * 192 ** -0.5 * U_BF16 / math.sqrt(3) * np.sqrt(((lat ** 2) @ (c ** 2).T + (rot ** 2) @ (kr ** 2).T).max(1)) + 2.0 ** -15
            assert_decode(b["out"], b["lse"], ref)
        lens = lens + accepted
        host.assign(lens)
        DevView(s).equals(host)


class DevView(DevTables):
    def __init__(self, s):
        self.table, self.held, self.stack, self.count = s.table, s.held, s.free, s.count


@gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_sparse_graphs_that_share_a_workspace(api, kv):
    """Two captured calls of other sizes on one workspace, replayed by turns and again: each as if it were alone."""
    ts = [Topics(api, [3000, 700], 1, 16, kv, 6, 1, 2, seed=1), Topics(api, [900, 64, 5000, 130], 2, 32, kv, 9, 1, 2, seed=2)]
    ds = [t.dev() for t in ts]
    want = [t.run(d) for t, d in zip(ts, ds)]
    ws = torch.empty(max(api.decode_sparse_workspace_size(len(t.lens), t.T, t.H, t.table.shape[1], t.keep) for t in ts), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got, graphs = [], []
    with torch.cuda.stream(stream):
        for t, d in zip(ts, ds):
            cu, out, lse = i32(t.cu), torch.empty_like(want[len(got)][0]), torch.empty_like(want[len(got)][1])
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                t.run(d, cu_q=cu, out=out, lse=lse, workspace=ws)
            got.append((out, lse, cu))
            graphs.append(g)
        for k in (0, 1, 1, 0, 1, 0, 0):
            got[k][0].fill_(float("nan"))
            graphs[k].replay()
            stream.synchronize()
            assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][1], want[k][1])


@gpu
def test_sparse_calls_on_two_streams(api):
    """Calls that overlap on two streams, each with its own workspace, given by the stream argument."""
    ts = [Topics(api, [64 * 90 + 5, 3000], 1, 64, "bf16", 8, 1, 2, seed=k) for k in range(2)]
    ds, want = [t.dev() for t in ts], []
    for t, d in zip(ts, ds):
        want.append(t.run(d))
    cus = [i32(t.cu) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for k in range(2):
            got[k].append(ts[k].run(ds[k], cu_q=cus[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


@gpu
def test_sparse_sees_inputs_that_copies_changed_between_calls(api):
    """Inputs rewritten between calls on one stream, by copies and by kernels, in the same places."""
    ts = [Topics(api, [64 * 30 + 5, 3000, 200], 2, 32, "bf16", 7, 1, 2, seed=k) for k in range(3)]
    ds = [t.dev() for t in ts]
    want = [t.run(d) for t, d in zip(ts, ds)]
    cu = i32(ts[0].cu)
    place = {k: torch.zeros((max(d[k].shape[0] for d in ds),) + v.shape[1:], dtype=v.dtype, device="cuda") for k, v in ds[0].items()}
    ws = torch.empty(api.decode_sparse_workspace_size(3, 6, 32, ts[0].table.shape[1], 7), dtype=torch.uint8, device="cuda")
    for rep in range(6):
        k = rep % 3
        for name, v in ds[k].items():
            place[name][:v.shape[0]].copy_(v)
        n = ds[k]["kv_cache"].shape[0]
        out, lse = ts[k].run({name: (v[:n] if name in ("kv_cache", "means") else v) for name, v in place.items()}, cu_q=cu, workspace=ws)
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


@gpu
def test_scores_and_choice_repeat_bit_for_bit(api):
    s = Scores([64 * 200 + 5, 9000, 700], 2, 128, seed=4)
    first = s.run(api).clone()
    for _ in range(5):
        assert torch.equal(s.run(api), first)


@gpu
@pytest.mark.parametrize("rows", [1, 128], ids=["few_candidates", "many"])
def test_means_read_tables_that_the_call_before_assigned(api, rows):
    """The means' launch follows the one that writes the block table, whose entries were -1 before."""
    B = 200
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = torch.randn((2 * B, 64, 576), generator=g, device="cuda").bfloat16()
    table, held = torch.full((B, 2), -1, dtype=torch.int32, device="cuda"), i32(np.zeros(B))
    free, count, err = i32(np.arange(2 * B)), i32([2 * B]), torch.zeros(1, dtype=torch.int32, device="cuda")
    none, full = i32(np.zeros(B)), i32(np.full(B, 128))
    means = torch.zeros((2 * B, 576), dtype=torch.bfloat16, device="cuda")

    def step():
        api.assign_blocks(table, held, none, free, count)
        api.assign_blocks(table, held, full, free, count)
        api.block_means(cache, table, full, means, rows=rows * B, dev_error=err)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        want = cache.double().mean(1).cpu().numpy()
        size = cache.double().abs().mean(1).cpu().numpy()
        ids = table.cpu().numpy()[:, 2 - max(1, rows // 64):].ravel()
        for _ in range(5):
            means.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = means.double().cpu().numpy()
            assert int(err) == 0
            assert (np.abs(got[ids] - want[ids]) <= U_BF16 * np.abs(want[ids]) + 64 * U_FP32 * size[ids]).all()


@gpu
def test_choice_reads_lengths_that_the_call_before_wrote(api):
    """A choice among the blocks that a choice left: its block table and lengths are what the launch before writes."""
    T, width, keep = 300, 400, 40
    g = torch.Generator(device="cuda").manual_seed(6)
    scores, again = torch.rand((T, width), generator=g, device="cuda"), torch.rand((T, keep), generator=g, device="cuda")
    blocks = torch.randperm(T * width, generator=g, device="cuda").int().view(T, width).contiguous()
    seq = i32(64 * width - np.arange(T) % 64)
    table, lens = torch.empty((T, keep), dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    table2, lens2 = torch.empty((T, 9), dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")

    def step():
        api.select_blocks(scores, blocks, seq, keep=keep, table=table, lens=lens)
        api.select_blocks(again, table, lens, keep=9, sinks=1, recent=2, table=table2, lens=lens2)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        want, want_lens = table2.clone(), lens2.clone()
        first, s = table.cpu().numpy(), again.cpu().numpy()
        for x in range(T):
            mid = sorted(1 + np.argsort(-s[x, 1:keep - 2], kind="stable")[:6])
            assert want[x].tolist() == [int(first[x, j]) for j in [0, *mid, keep - 2, keep - 1]]
            assert int(want_lens[x]) == 8 * 64 + (int(seq[x]) - 1) % 64 + 1
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(5):
            for t in (table, lens, table2, lens2):
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(table2, want) and torch.equal(lens2, want_lens)
