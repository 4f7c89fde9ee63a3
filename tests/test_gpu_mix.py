"""Token mixing (q4gemv_kv_append, q4gemv_attn_paged, q4gemv_linattn) through
the binding against plain 64-bit forms.

Tolerances, from the arithmetic (u = half a step of the 16-bit type):
  append  an output is rounded once (u of it) from 32-bit products whose
          cosines and sines are off by a few 2^-24 (argument and function), so
          u |y| + 2^-20 (|a| + |b|) amp.
  attend  scores are 32-bit sums of head_dim products (at most head_dim 2^-23
          of their magnitudes, a factor on the weights), weights may be rounded
          once to the type before they meet v (u each; for f16 also 2^-25 of the
          largest weight each, its subnormals), sums of up to len terms in 32
          bits, and one final rounding:
          (u + 2 head_dim 2^-23 mags + 2^-18) A + len 2^-25 max|v| + u |o|, with A the
          weighted magnitudes of v (2^-18: exp2 and the sums of up to 2^11
          steps of 2^-23 in tiles).
  linear  state: 32-bit sums of a token's terms, at most (tokens + 64) 2^-22 of
          their magnitudes.  out: each term (state times query, or score times
          value) has one operand that is rounded once to the type, a factor
          1 + d with |d| <= u: together at most u A, A the terms' magnitudes
          (binary16 is given 2^-10 = 2 u, as before the operands' type was the
          tensors'; bfloat16 u = 2^-8); the same sums, and u |o| for the output.
"""
import os
import subprocess
import sys

import pytest

from tests import mix_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import q4_quantized_decode_b200 as q4  # noqa: E402

DTYPES = [torch.float16, torch.bfloat16]
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def eng():
    e = q4.Q4Gemv(0)
    yield e
    e.close()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def gpu_pool(x):
    """The pool on the GPU with the same strides (a permuted view stays one)."""
    if x.is_contiguous():
        return x.to(DEV)
    return x.transpose(1, 2).to(DEV).transpose(1, 2)


def close(got, want, tol, what):
    got = got.detach().to("cpu", torch.float64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} over the tolerance at {int(over.argmax())}"


# ---- append -----------------------------------------------------------------

class AppendCase:
    def __init__(self, new, ctx, hq, hkv, dim, page, dtype, seed=0, head_major=False, fused=True):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.dtype, self.dim, self.hq, self.hkv = new, dtype, dim, hq, hkv
        self.length = [n + c for n, c in zip(new, ctx)]
        self.rows = sum(new)
        self.table, pool = ref.table_of(self.length, page, gen)
        self.k0 = ref.paged(pool, page, hkv, dim, dtype, gen, head_major)
        self.v0 = ref.paged(pool, page, hkv, dim, dtype, gen, head_major)
        w = (hq + 2 * hkv) * dim
        qkv = torch.randn(self.rows, w, generator=gen).to(dtype)
        cut = lambda x, a, h: x[:, a * dim:(a + h) * dim].unflatten(1, (h, dim))  # noqa: E731
        self.q, self.k, self.v = cut(qkv, 0, hq), cut(qkv, hq, hkv), cut(qkv, hq + hkv, hkv)
        g = qkv.to(DEV)
        self.gq, self.gk, self.gv = cut(g, 0, hq), cut(g, hq, hkv), cut(g, hq + hkv, hkv)
        if not fused:
            self.gq, self.gk, self.gv = (x.contiguous() for x in (self.gq, self.gk, self.gv))
        self.cache = q4.PagedKV(gpu_pool(self.k0), gpu_pool(self.v0), self.table.to(DEV))
        self.start, self.glen = ints(starts(new)), ints(self.length)
        self.pos = torch.tensor([p for n, l in zip(new, self.length) for p in range(l - n, l)], dtype=torch.int64)
        self.seq = [s for s, n in enumerate(new) for _ in range(n)]
        self.page = page

    def check(self, qo, freqs, interleaved=False, amp=1.0, pos=None):
        pos = self.pos if pos is None else pos
        u, t = ref.half_step(self.dtype), ref.tiny(self.dtype)
        for name, x, got in (("q", self.q, qo), ("k", self.k, None)):
            want, mag = ref.rotate(x, pos, freqs, interleaved, amp)
            if got is None:
                at = self.pos
                pg = self.table[self.seq, at // self.page].long()
                kd = self.cache.k.cpu()
                close(kd[pg, at % self.page], want, u * want.abs() + 2.0 ** -20 * mag + t, "k")
                rest = torch.ones(kd.shape[:2], dtype=torch.bool)
                rest[pg, at % self.page] = False
                assert torch.equal(kd[rest], self.k0[rest]), "slots of no new token changed"
                vd = self.cache.v.cpu()
                assert torch.equal(vd[pg, at % self.page], self.v)
                assert torch.equal(vd[rest], self.v0[rest])
            elif got is not False:
                close(got, want, u * want.abs() + 2.0 ** -20 * mag + t, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 64), (96, 96), (80, 32), (256, 64), (8, 8), (64, 20),
                                     (128, 0), (72, 2), (64, 34)])
def test_append_layouts(eng, dtype, interleaved, dim, rot):
    c = AppendCase([3, 1, 0, 17], [0, 31, 5, 100], 6, 2, dim, 16, dtype, seed=dim + rot)
    st, f = q4.q4gemv_rope_freqs(q4.ROPE_PLAIN, rot, 10000.0)
    freqs = torch.tensor(f, dtype=torch.float64, device=DEV) if rot else None
    qo = eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=c.gq, freqs=freqs, interleaved=interleaved, amp=1.25)
    assert eng.sync_status() == q4.Q4_OK
    c.check(qo, f, interleaved, 1.25 if rot else 1.0)


@pytest.mark.parametrize("page,head_major", [(1, False), (7, True), (24, False), (64, True), (1000, False)])
def test_append_pages_and_layouts(eng, page, head_major):
    c = AppendCase([5, 40, 1], [99, 0, 1000], 8, 8, 64, page, torch.float16, seed=page, head_major=head_major, fused=False)
    f = eng.rope_freqs(64)
    qo = eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=c.gq, freqs=f)
    assert eng.sync_status() == q4.Q4_OK
    c.check(qo, f.cpu())


@pytest.mark.parametrize("kind,factor", [(q4.ROPE_PLAIN, 1.0), (q4.ROPE_LINEAR, 4.0), (q4.ROPE_BY_PARTS, 16.0)])
def test_append_far_positions(eng, kind, factor):
    """Positions of a million: the angle has to be taken in 64 bits."""
    c = AppendCase([2, 9], [0, 50], 4, 1, 128, 32, torch.float16, seed=3)
    f = eng.rope_freqs(128, base=1e6, kind=kind, factor=factor, trained=32768.0)
    pos = torch.tensor([0, 1] + [999_983 + 7 * i for i in range(8)] + [2**31 - 1], dtype=torch.int64)
    qo = eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=c.gq, freqs=f, pos=ints(pos.tolist()))
    assert eng.sync_status() == q4.Q4_OK
    c.check(qo, f.cpu(), pos=pos)


def test_append_in_place_and_without_queries(eng):
    c = AppendCase([6], [20], 5, 1, 64, 16, torch.bfloat16, seed=4, fused=False)
    f = eng.rope_freqs(48)
    q = c.gq.clone()
    assert eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=q, q_out=q, freqs=f, interleaved=True) is q
    c.check(q, f.cpu(), True)
    c = AppendCase([6], [20], 5, 1, 64, 16, torch.bfloat16, seed=5)
    assert eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, freqs=f) is None
    c.check(False, f.cpu())
    assert eng.sync_status() == q4.Q4_OK


def test_append_leaves_other_rows(eng):
    """Rows behind the last sequence are neither read nor written."""
    c = AppendCase([4, 2], [3, 0], 2, 1, 64, 8, torch.float16, seed=6, fused=False)
    start = ints([0, 4, 5])                              # the last row is nobody's
    length = ints([7, 1])
    out = torch.full_like(c.gq, 7.0)
    eng.kv_append(c.cache, start, length, c.gk, c.gv, q=c.gq, q_out=out, freqs=eng.rope_freqs(64))
    assert eng.sync_status() == q4.Q4_OK
    assert (out[5] == 7.0).all() and not (out[:5] == 7.0).all()


def test_append_infinite_values_pass_where_not_rotated(eng):
    c = AppendCase([1], [0], 1, 1, 64, 8, torch.float16, seed=7, fused=False)
    for il in (False, True):
        q = c.gq.clone()
        q[0, 0, 20] = float("nan")
        q[0, 0, 23] = float("inf")
        out = eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=q, freqs=eng.rope_freqs(20), interleaved=il)
        assert torch.isnan(out[0, 0, 20]) and torch.isinf(out[0, 0, 23])
        assert torch.isfinite(out[0, 0, :20]).all() and torch.equal(out[0, 0, 24:], q[0, 0, 24:])


def test_append_bad_pages_are_reported(eng):
    c = AppendCase([2, 3], [0, 14], 2, 1, 64, 8, torch.float16, seed=8)
    k0 = c.cache.k.clone()
    c.cache.table[0, 0] = c.k0.shape[0]                  # past the pool
    c.cache.table[1, 2] = -5
    qo = eng.kv_append(c.cache, c.start, c.glen, c.gk, c.gv, q=c.gq, freqs=eng.rope_freqs(64))
    assert eng.sync_status() == q4.Q4_EINDEX
    assert eng.sync_status() == q4.Q4_OK
    want, mag = ref.rotate(c.q, c.pos, eng.rope_freqs(64).cpu())
    close(qo, want, 2.0 ** -11 * want.abs() + 2.0 ** -20 * mag + 2.0 ** -25, "q")
    changed = (c.cache.k != k0).any(-1).any(-1)          # rows 14, 15 of sequence 1 only (place 16 is in the bad page)
    assert int(changed.sum()) == 2
    # a length under the new tokens' count: negative places
    eng.kv_append(c.cache, c.start, ints([1, 17]), c.gk, c.gv)
    assert eng.sync_status() == q4.Q4_EINDEX
    # past the table's columns
    eng.kv_append(c.cache, c.start, ints([2, 8 * c.table.shape[1] + 3]), c.gk, c.gv)
    assert eng.sync_status() == q4.Q4_EINDEX


# ---- attend -----------------------------------------------------------------

# Columns of the page table: a table that could hold long contexts sends
# sequences of more than 64 rows to the tensor-core kernel.
WIDE = 1 << 14


class AttendCase:
    def __init__(self, new, length, hq, hkv, dim, page, dtype, seed=0, head_major=False, poison=True, amp=1.0,
                 cols=0):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.length, self.hq, self.hkv, self.dim, self.dtype = new, length, hq, hkv, dim, dtype
        self.rows = sum(new)
        self.table, pool = ref.table_of(length, page, gen, cols=cols)
        self.k, self.v = (ref.paged(pool, page, hkv, dim, dtype, gen, head_major) for _ in range(2))
        if poison:                                       # what no token has written is NaN
            used = torch.zeros(pool, page, dtype=torch.bool)
            for s, l in enumerate(length):
                j = torch.arange(l)
                used[self.table[s, j // page].long(), j % page] = True
            self.k[~used] = float("nan")
            self.v[~used] = float("nan")
        self.q = (amp * torch.randn(self.rows, hq, dim, generator=gen)).to(dtype)
        self.cache = q4.PagedKV(gpu_pool(self.k), gpu_pool(self.v), self.table.to(DEV))
        self.gq, self.start, self.glen = self.q.to(DEV), ints(starts(new)), ints(length)

    def run(self, eng, **kw):
        return eng.attn_paged(self.cache, self.start, self.glen, self.gq, **kw)

    def check(self, out, scale=None, causal=True, window=0, seqs=None, heads=None):
        scale = self.dim ** -0.5 if scale is None else scale
        u = ref.half_step(self.dtype)
        out = out.cpu()
        at = starts(self.new)
        for s, (n, l) in enumerate(zip(self.new, self.length)):
            if n == 0 or (seqs is not None and s not in seqs):
                continue
            for h in range(self.hq) if heads is None else heads:
                kv = h // (self.hq // self.hkv)
                k, v = (ref.gather(x, self.table, s, l, kv) for x in (self.k, self.v))
                o, a, mags = ref.attend(self.q[at[s]:at[s + 1], h], k, v, l - n, scale, causal, window)
                top = torch.nan_to_num(v.double(), 0.0, 0.0, 0.0).abs().amax() if l else 0.0
                tol = (u + 2 * self.dim * 2.0 ** -23 * mags[:, None] + 2.0 ** -18) * a + \
                    l * 2.0 ** -25 * top + u * o.abs() + ref.tiny(self.dtype)
                close(out[at[s]:at[s + 1], h], o, tol, f"sequence {s}, head {h}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,dim", [(5, 1, 128), (8, 8, 64), (8, 2, 64), (6, 2, 128), (4, 1, 256), (3, 3, 96),
                                        (2, 1, 8), (20, 1, 80), (40, 2, 64), (4, 2, 248)])
def test_attend_single_tokens(eng, dtype, hq, hkv, dim):
    c = AttendCase([1] * 6, [1, 2, 31, 64, 257, 700], hq, hkv, dim, 16, dtype, seed=hq + dim)
    out = c.run(eng, max_new=1)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page,head_major", [(1, False), (5, False), (16, True), (24, False), (100, True), (1024, False)])
def test_attend_pages(eng, cols, dtype, page, head_major):
    c = AttendCase([1, 3, 70], [300, 77, 211], 4, 2, 64, page, dtype, seed=page, head_major=head_major, cols=cols)
    out = c.run(eng, max_new=70)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,length", [([169], [169]), ([128, 0, 1, 33], [128, 40, 513, 1000]), ([200], [1300]),
                                        ([257, 64], [257, 65]), ([600], [600])])
@pytest.mark.parametrize("hq,hkv,dim", [(5, 1, 128), (4, 4, 64), (2, 1, 256), (3, 1, 72)])
def test_attend_chunks(eng, cols, dtype, new, length, hq, hkv, dim):
    c = AttendCase(new, length, hq, hkv, dim, 16, dtype, seed=sum(new) + dim, cols=cols)
    out = c.run(eng, max_new=max(new))
    assert eng.sync_status() == q4.Q4_OK
    c.check(out)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 7), (True, 130), (True, 100000), (False, 0), (False, 40)])
@pytest.mark.parametrize("new,length", [([1, 1], [500, 3]), ([4, 5], [260, 9]), ([150], [400])])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_masks(eng, cols, causal, window, new, length, dim):
    c = AttendCase(new, length, 4, 2, dim, 24, torch.float16, seed=window + sum(new), cols=cols)
    out = c.run(eng, causal=causal, window=window, max_new=max(new))
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, causal=causal, window=window)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("max_new", [1, 5, 1000])
def test_attend_max_new_is_only_a_hint(eng, cols, max_new):
    c = AttendCase([1, 150, 0, 9], [900, 170, 8, 300], 6, 2, 128, 16, torch.float16, seed=9, cols=cols)
    out = c.run(eng, max_new=max_new)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 200])
def test_attend_rows_that_see_nothing(eng, cols, dim, new):
    """A length under the count of the new tokens: the first rows stand before
    the cache's beginning and see nothing; length 0: no row sees anything."""
    c = AttendCase([new, new], [new - 2, 0], 2, 1, dim, 16, torch.float16, seed=dim, cols=cols)
    out = c.run(eng, max_new=new)
    assert eng.sync_status() == q4.Q4_OK
    assert (out[:2] == 0).all() and (out[new:] == 0).all()
    c.check(out)


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [4, 180])
def test_attend_non_finite_values_of_unseen_tokens(eng, cols, bad, dim, new):
    """A later token of the chunk, or one before the window, holds NaN or Inf in
    its key and value: rows that do not see it are unaffected; rows that see it
    are not finite."""
    c = AttendCase([new], [new + 50], 2, 1, dim, 16, torch.float16, seed=dim + new, cols=cols)
    j = new + 50 - 2                                     # the last but one token
    pg, at = int(c.table[0, j // 16]), j % 16
    for pool in (c.k, c.v, c.cache.k, c.cache.v):
        pool[pg, at, 0, 3] = bad
    out = c.run(eng, max_new=new)
    assert eng.sync_status() == q4.Q4_OK
    assert torch.isfinite(out[:new - 2]).all()
    if bad != bad:
        assert torch.isnan(out[new - 2:]).all()
    clean = AttendCase([new], [new + 50], 2, 1, dim, 16, torch.float16, seed=dim + new, cols=cols)
    same = clean.run(eng, max_new=new)
    clean.check(same)
    same[:new - 2] = out[:new - 2]
    clean.check(same)
    # before the window
    w = 40
    c2 = AttendCase([new], [new + 50], 2, 1, dim, 16, torch.float16, seed=dim + new, cols=cols)
    pg, at = int(c2.table[0, 0]), 2
    for pool in (c2.k, c2.v, c2.cache.k, c2.cache.v):
        pool[pg, at, 0, :] = bad
    out = c2.run(eng, max_new=new, window=w)
    assert eng.sync_status() == q4.Q4_OK
    c2.check(out, window=w)


@pytest.mark.parametrize("cols", [0, WIDE])
def test_attend_large_scores(eng, cols):
    """Scores of hundreds: one token takes all the weight; the running maximum
    has to follow."""
    for dim, new in ((64, 1), (128, 2), (128, 140), (64, 140), (256, 3)):
        c = AttendCase([new], [600], 4, 2, dim, 16, torch.float16, seed=dim, amp=30.0, cols=cols)
        out = c.run(eng, max_new=new)
        c.check(out)
        out = c.run(eng, max_new=new, scale=0.0)
        c.check(out, scale=0.0)
        out = c.run(eng, max_new=new, scale=-0.02)
        c.check(out, scale=-0.02)
    assert eng.sync_status() == q4.Q4_OK


@pytest.mark.parametrize("cols", [0, WIDE])
def test_attend_strides_and_rows_of_no_sequence(eng, cols):
    for new in ([1, 2], [90, 40]):
        c = AttendCase(new, [70 + new[0], 200], 4, 2, 64, 16, torch.bfloat16, seed=11, cols=cols)
        rows = c.rows
        wide = torch.full((rows + 3, 4 * 64 + 24), 5.0, dtype=c.dtype, device=DEV)
        q = wide.clone()[:, :256].unflatten(1, (4, 64))
        q[:rows] = c.gq
        out = wide[:, 8:264].unflatten(1, (4, 64))
        got = eng.attn_paged(c.cache, c.start, c.glen, q, out=out, max_new=max(new))
        assert got is out and eng.sync_status() == q4.Q4_OK
        c.check(out[:rows])
        assert (out[rows:] == 5.0).all() and (wide[:, :8] == 5.0).all() and (wide[:, 264:] == 5.0).all()


def test_attend_shared_pages(eng):
    """Two sequences with the same prefix pages."""
    c = AttendCase([1, 2], [64, 64], 4, 2, 64, 16, torch.float16, seed=12, poison=False)
    c.table[1, :3] = c.table[0, :3]
    c.cache.table.copy_(c.table)
    c.check(c.run(eng, max_new=2))
    assert eng.sync_status() == q4.Q4_OK


@pytest.mark.parametrize("cols", [0, WIDE])
@pytest.mark.parametrize("new", [1, 100])
def test_attend_bad_pages_are_left_out(eng, cols, new):
    c = AttendCase([new, new], [200, 300], 4, 2, 128, 16, torch.float16, seed=13, cols=cols)
    good = c.cache.table.clone()
    c.cache.table[0, 3] = 10 ** 6
    c.cache.table[0, 4] = -1
    out = c.run(eng, max_new=new)
    assert eng.sync_status() == q4.Q4_EINDEX
    assert torch.isfinite(out).all()
    c.check(out, seqs=[1])
    # the first sequence as if those 32 tokens were not there
    u = 2.0 ** -11
    for h in range(4):
        k, v = (ref.gather(x, c.table, 0, 200, h // 2) for x in (c.k, c.v))
        keep = torch.cat((torch.arange(48), torch.arange(80, 200)))
        o, a, mags = ref.attend(c.q[:new, h], k[keep], v[keep], 200 - new - 32, 128 ** -0.5)
        tol = (u + 256 * 2.0 ** -23 * mags[:, None] + 2.0 ** -18) * a + 200 * 2.0 ** -25 * 6 + u * o.abs() + 2.0 ** -25
        close(out[:new, h], o, tol, "without the bad pages")
    c.cache.table.copy_(good)
    c.check(c.run(eng, max_new=new))
    # a length past the table's columns
    eng.attn_paged(c.cache, c.start, ints([200, 16 * c.table.shape[1] + 40]), c.gq, max_new=new)
    assert eng.sync_status() == q4.Q4_EINDEX


@pytest.mark.parametrize("cols", [0, WIDE])
def test_attend_is_deterministic_and_follows_a_graph(eng, cols):
    """A captured call replayed after the lengths, tables and queries changed."""
    for new in (1, 120):
        c = AttendCase([new, new, new], [900, 130, 350], 8, 2, 128, 16, torch.float16, seed=14, cols=cols)
        a, b = c.run(eng, max_new=new), c.run(eng, max_new=new)
        assert torch.equal(a, b)
        out = torch.zeros_like(c.gq)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            eng.attn_paged(c.cache, c.start, c.glen, c.gq, out=out, max_new=new)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
        d = AttendCase([new, new, new], [500, 700, 121], 8, 2, 128, 16, torch.float16, seed=15, cols=cols)
        n, cols = d.cache.k.shape[0], d.table.shape[1]
        assert n <= c.cache.k.shape[0] and cols <= c.table.shape[1]
        c.glen.copy_(d.glen)
        c.gq.copy_(d.gq)
        c.cache.table.fill_(-1)
        c.cache.table[:, :cols].copy_(d.cache.table)
        c.cache.k[:n].copy_(d.cache.k)
        c.cache.v[:n].copy_(d.cache.v)
        g.replay()
        torch.cuda.synchronize()
        d.check(out)
        assert eng.sync_status() == q4.Q4_OK


def test_attend_long_context_offsets(eng):
    """A pool of more than 2^31 elements: the far pages' offsets pass 32 bits."""
    page, hkv, dim = 64, 8, 128
    pool = 2 ** 31 // (page * hkv * dim) + 40
    k = torch.zeros(pool, page, hkv, dim, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    gen = torch.Generator().manual_seed(1)
    for new in (1, 80):
        table = torch.full((1, WIDE), -1, dtype=torch.int32)
        table[0, :7] = torch.arange(pool - 7, pool, dtype=torch.int32).flip(0)
        kk, vv = (torch.randn(7 * page, hkv, dim, generator=gen).half() for _ in range(2))
        k[pool - 7:] = kk.view(7, page, hkv, dim).to(DEV)
        v[pool - 7:] = vv.view(7, page, hkv, dim).to(DEV)
        q = torch.randn(new, 2 * hkv, dim, generator=gen).half()
        cache = q4.PagedKV(k, v, table.to(DEV))
        out = eng.attn_paged(cache, ints([0, new]), ints([400]), q.to(DEV), max_new=new).cpu()
        assert eng.sync_status() == q4.Q4_OK
        kc, vc = (x.view(7, page, hkv, dim).flip(0).reshape(-1, hkv, dim)[:400] for x in (kk, vv))
        for h in (0, 15):
            o, a, mags = ref.attend(q[:, h], kc[:, h // 2], vc[:, h // 2], 400 - new, dim ** -0.5)
            tol = (2.0 ** -11 + 256 * 2.0 ** -23 * mags[:, None] + 2.0 ** -18) * a + 400 * 2.0 ** -25 * 6 + \
                2.0 ** -11 * o.abs() + 2.0 ** -25
            close(out[:, h], o, tol, f"head {h}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,page", [(136, 16), (200, 24), (256, 5), (256, 64), (256, 1024)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0), (False, 33)])
def test_attend_chunks_of_wide_heads(eng, dtype, dim, page, causal, window):
    """Head sizes past 128 on the tensor-core kernel: units of 128 rows, whole
    and in pieces, of ragged sequences."""
    c = AttendCase([70, 0, 301, 129], [70, 9, 640, 2500], 4, 2, dim, page, dtype, seed=dim + page, cols=WIDE,
                   head_major=page == 64)
    out = c.run(eng, max_new=301, causal=causal, window=window)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, causal=causal, window=window)
    assert torch.equal(out, c.run(eng, max_new=301, causal=causal, window=window))


@pytest.mark.parametrize("scale", [None, 0.0, -0.02, 3.0])
def test_attend_wide_heads_large_scores(eng, scale):
    for new, length in ((140, 600), (1000, 1400)):
        c = AttendCase([new], [length], 3, 1, 256, 16, torch.float16, seed=new, amp=30.0, cols=WIDE)
        c.check(c.run(eng, scale=scale), scale=scale)
    assert eng.sync_status() == q4.Q4_OK


def test_attend_wide_heads_bad_pages(eng):
    c = AttendCase([150, 150], [400, 300], 4, 2, 256, 16, torch.float16, seed=17, cols=WIDE)
    c.cache.table[0, 3] = 10 ** 6
    out = c.run(eng)
    assert eng.sync_status() == q4.Q4_EINDEX
    assert torch.isfinite(out).all()
    c.check(out, seqs=[1])
    keep = torch.cat((torch.arange(48), torch.arange(64, 400)))
    for h in range(4):
        k, v = (ref.gather(x, c.table, 0, 400, h // 2) for x in (c.k, c.v))
        o, a, mags = ref.attend(c.q[:150, h], k[keep], v[keep], 400 - 150 - 16, 1 / 16)
        tol = (2.0 ** -11 + 512 * 2.0 ** -23 * mags[:, None] + 2.0 ** -18) * a + 400 * 2.0 ** -25 * 6 + \
            2.0 ** -11 * o.abs() + 2.0 ** -25
        close(out[:150, h], o, tol, "without the bad page")


@pytest.mark.parametrize("new", [1, 200])
def test_attend_places_near_the_end_of_32_bits(eng, new):
    """A table of 2^31 places (one page, over and over) and a length that
    reaches their end: what lies from place 2^31 - 2^25 on is left out and told.
    Keys and queries are zeros, so all weights are 1 and every output is the one
    value.  A piece (a CTA's part, at least 148 of them) has under 2^24 tokens, so
    its sums of ones are exact, and its sums of 1.5 a tile (multiples of 8 under
    2^25) are too; joining under 2^10 pieces in 32 bits is off by less than
    2^-13, the output's rounding by 2^-11 of the value: 2^-10 together."""
    page = 1 << 20
    k = torch.zeros(1, page, 1, 8, dtype=torch.float16, device=DEV)
    v = torch.full_like(k, 1.5)
    cache = q4.PagedKV(k, v, torch.zeros(1, 2 ** 31 // page, dtype=torch.int32, device=DEV))
    q = torch.zeros(new, 1, 8, dtype=torch.float16, device=DEV)
    out = eng.attn_paged(cache, ints([0, new]), ints([2 ** 31 - 1]), q)
    assert eng.sync_status() == q4.Q4_EINDEX
    assert (out.float() - 1.5).abs().max().item() <= 1.5 * 2.0 ** -10


def test_attend_more_rows_than_32_bits_are_refused(eng):
    """2^24 rows of 1024 query heads to a key head: refused before anything is read."""
    c = AttendCase([1], [20], 1, 1, 8, 16, torch.float16, seed=35)
    a = c.gq.data_ptr()
    st = q4.q4gemv_attn_paged(eng.h, c.cache.ref, 1 << 24, 1, c.start.data_ptr(), c.glen.data_ptr(), 1, a, 8192, 1024,
                              a + 16, 8192, 1.0, 1, 0, None)
    assert st == q4.Q4_ESHAPE and eng.sync_status() == q4.Q4_OK


# ---- linear -----------------------------------------------------------------

class LinearCase:
    def __init__(self, new, hk, hv, dk, dv, dtype, seed=0, fixed=False, slots=None, rate=(-1.0, -8.0)):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.hk, self.hv, self.dk, self.dv, self.dtype = new, hk, hv, dk, dv, dtype
        rows = self.rows = sum(new)
        n = len(new)
        self.slots = torch.randperm(n + 1, generator=gen)[:n].to(torch.int32) if slots is None else slots
        qkv = torch.randn(rows, 2 * hk * dk + hv * dv, generator=gen)
        qkv[:, :2 * hk * dk] *= dk ** -0.5
        qkv = qkv.to(dtype)
        cut = lambda x: (x[:, :hk * dk].unflatten(1, (hk, dk)), x[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk)),  # noqa: E731
                         x[:, 2 * hk * dk:].unflatten(1, (hv, dv)))
        self.q, self.k, self.v = cut(qkv)
        self.gq, self.gk, self.gv = cut(qkv.to(DEV))
        r = 2.0 ** (rate[0] + (rate[1] - rate[0]) * torch.rand(1 if fixed else rows, hv, generator=gen))
        self.g = (-r).expand(rows, hv) if fixed else -r
        self.gg = (-r).to(DEV).expand(rows, hv) if fixed else (-r).to(DEV)
        self.state = torch.randn(n + 1, hv, dk, dv, generator=gen)
        self.start = ints(starts(new))

    def run(self, eng, state=None, **kw):
        kw.setdefault("slots", self.slots.to(DEV))
        kw.setdefault("max_new", max([1] + self.new))
        return eng.linattn(self.gq, self.gk, self.gv, self.gg, self.start,
                           self.state.to(DEV) if state is None else state, **kw)

    def check(self, out, state, scale=1.0, zero=False, seqs=None, heads=None):
        u = ref.half_step(self.dtype)
        out, state = out.cpu(), state.cpu()
        at = starts(self.new)
        for s, n in enumerate(self.new):
            if seqs is not None and s not in seqs:
                continue
            sl = slice(at[s], at[s + 1])
            for h in range(self.hv) if heads is None else heads:
                hk = h // (self.hv // self.hk)
                s0 = self.state[self.slots[s], h]
                o, S, ao, A = ref.linear(self.q[sl, hk], self.k[sl, hk], self.v[sl, h], self.g[sl, h],
                                         torch.zeros_like(s0) if zero else s0, scale)
                sums = (n + 64) * 2.0 ** -22
                close(state[self.slots[s], h], S, sums * A, f"state {s}, head {h}")
                close(out[sl, h], o, (max(u, 2.0 ** -10) + sums) * ao + u * o.abs() + ref.tiny(self.dtype),
                      f"sequence {s}, head {h}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 128, 128), (2, 6, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128),
                                         (1, 1, 8, 8), (1, 2, 72, 40), (1, 1, 256, 256), (3, 3, 136, 24)])
def test_linear_single_tokens(eng, dtype, hk, hv, dk, dv):
    c = LinearCase([1, 1, 0, 2, 1], hk, hv, dk, dv, dtype, seed=dk + dv)
    out, state = c.run(eng, scale=0.5)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, state, scale=0.5)
    unused = (set(range(6)) - set(c.slots.tolist())).pop()
    assert torch.equal(state[unused].cpu(), c.state[unused])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("new", [[64], [65, 0, 1, 63], [130, 17], [300], [5, 128, 127]])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 128), (2, 2, 64, 64), (1, 1, 64, 128), (1, 1, 24, 40), (1, 1, 256, 72)])
def test_linear_prompts(eng, dtype, fixed, new, hk, hv, dk, dv):
    c = LinearCase(new, hk, hv, dk, dv, dtype, seed=sum(new) + dk, fixed=fixed)
    out, state = c.run(eng)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, state)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[1500], [1024, 0, 70, 801], [777, 64]])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 128), (1, 1, 64, 64), (1, 1, 256, 72)])
def test_linear_long_prompts_in_segments(eng, dtype, new, hk, hv, dk, dv):
    """Few heads and long prompts: sequences run as parallel segments, some of
    them without tokens; the state is updated in place."""
    c = LinearCase(new, hk, hv, dk, dv, dtype, seed=sum(new) + dv, rate=(-4.0, -12.0))
    state = c.state.to(DEV)
    out, end = c.run(eng, state=state)
    assert end is state and eng.sync_status() == q4.Q4_OK
    c.check(out, state)
    zero = torch.full_like(state, 9.0)
    out, _ = eng.linattn(c.gq, c.gk, c.gv, c.gg, c.start, None, state_out=zero, slots=c.slots.to(DEV), max_new=max(new))
    c.check(out, zero, zero=True)
    again, _ = c.run(eng, max_new=1 << 20)               # another cut
    c.check(again, c.run(eng, max_new=64)[1])


def test_linear_segments_pass_non_finite_states_on(eng):
    c = LinearCase([1400], 1, 2, 64, 64, torch.float16, seed=30)
    out0, _ = c.run(eng)
    c.gv = c.gv.clone()
    c.gv[700, 0, 5] = float("nan")
    out, state = c.run(eng)
    assert eng.sync_status() == q4.Q4_OK
    mixed = out0.clone()
    mixed[:700] = out[:700]
    mixed[:, 1] = out[:, 1]
    mixed[:, 0, :5] = out[:, 0, :5]
    ref_state = c.run(eng)[1].clone()
    assert torch.isnan(out[700:, 0, 5]).all() and torch.isnan(ref_state[c.slots[0], 0, :, 5]).all()
    clean = LinearCase([1400], 1, 2, 64, 64, torch.float16, seed=30)
    clean.check(mixed, clean.run(eng)[1])


@pytest.mark.parametrize("rate", [(3.0, 7.0), (-14.0, -20.0)])
def test_linear_strong_and_weak_decays(eng, rate):
    """Decays of e^-8 to e^-128 a token (differences of running sums lose all
    digits; a chunk's product underflows) and of nearly one."""
    for new in ([1, 3], [200, 70]):
        c = LinearCase(new, 1, 2, 64, 64, torch.float16, seed=21, rate=rate)
        out, state = c.run(eng)
        assert eng.sync_status() == q4.Q4_OK
        c.check(out, state)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kq,vv", [(2.0 ** -12, 1.0), (200.0, 100.0), (2.0 ** -6, 2.0 ** -9), (30.0, 2.0 ** -10)])
def test_linear_magnitudes(eng, dtype, kq, vv):
    """Keys, queries and values far from 1, and changing from chunk to chunk:
    the state keeps 32 bits' worth and nothing overflows on the way."""
    c = LinearCase([200, 5], 1, 2, 64, 64, dtype, seed=27)
    grow = torch.ones(c.rows, 1, 1)
    grow[64:128] = 8.0
    grow[128:] = 0.25
    c.q, c.k, c.v = (c.q.float() * 8 * kq).to(dtype), (c.k.float() * 8 * kq * grow).to(dtype), (c.v.float() * vv).to(dtype)
    c.state = c.state * (kq * vv)
    c.gq, c.gk, c.gv = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV)
    scale = 1.0 / (kq * kq * vv * 64)                    # outputs inside the type's range
    out, state = c.run(eng, scale=scale)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, state, scale=scale)


def test_linear_values_past_the_tensor_range(eng):
    """bfloat16 magnitudes of 2^35 in one chunk (run token by token), ordinary
    ones before and behind."""
    c = LinearCase([200], 1, 1, 64, 128, torch.bfloat16, seed=28)
    big = torch.ones(c.rows, 1, 1)
    big[70:75] = 2.0 ** 35
    c.v = (c.v.float() * big).to(torch.bfloat16)
    c.gv = c.v.to(DEV)
    out, state = c.run(eng)
    assert eng.sync_status() == q4.Q4_OK
    c.check(out, state)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "g"])
def test_linear_non_finite_tokens_reach_only_later_rows(eng, bad, what):
    if what == "g" and bad > 0:
        bad = float("nan")
    c = LinearCase([150, 20], 1, 2, 64, 64, torch.float16, seed=29)
    out0, state0 = c.run(eng)
    x = {"q": c.gq, "k": c.gk, "v": c.gv, "g": c.gg}[what].clone()
    if what == "g":
        x[100, 0] = bad
        c.gg = x
    else:
        x[100, 0, 5] = bad
        setattr(c, "g" + what, x)
    out, state = c.run(eng)
    assert eng.sync_status() == q4.Q4_OK
    clean = out0.clone()
    clean[:100] = out[:100]
    clean[150:] = out[150:]
    clean[:, 1] = out[:, 1] if what in ("v", "g") else clean[:, 1]      # the other value head
    c.check(clean, state0)
    hit = out[100:150, 0, 5] if what == "v" else out[100:150, 0]
    assert not torch.isfinite(out[100, 0]).all()
    if what != "q":
        assert not torch.isfinite(hit).any()
    else:
        keep = out.clone()
        keep[100] = out0[100]
        c.check(keep, state)


def test_linear_decay_of_minus_infinity_clears(eng):
    for new in ([3], [150]):
        c = LinearCase(new, 1, 1, 64, 64, torch.float16, seed=22)
        at = new[0] // 2
        c.g = c.g.clone()
        c.g[at] = -float("inf")
        c.gg[at] = -float("inf")
        out, state = c.run(eng)
        assert eng.sync_status() == q4.Q4_OK
        c.check(out, state)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dv", [8, 72, 128, 200])
def test_linear_prompts_write_their_rows_only(eng, dtype, dv):
    """Whole chunks of outputs leave in boxes: a strided output with columns
    around the heads and rows before, between and behind the sequences keeps
    what it had there."""
    c = LinearCase([300, 0, 128, 131], 1, 2, 64, dv, dtype, seed=dv)
    rows, w = c.rows, 2 * dv
    wide = torch.full((rows + 150, w + 24), 3.0, dtype=dtype, device=DEV)
    out = wide[:, 16:16 + w].unflatten(1, (2, dv))
    pad = lambda x: torch.cat((x, x.new_full((150,) + x.shape[1:], float("nan"))))  # noqa: E731
    got, state = eng.linattn(pad(c.gq), pad(c.gk), pad(c.gv), pad(c.gg), c.start, c.state.to(DEV),
                             slots=c.slots.to(DEV), out=out, max_new=300)
    assert eng.sync_status() == q4.Q4_OK
    c.check(got[:rows], state)
    assert (wide[rows:] == 3.0).all() and (wide[:, :16] == 3.0).all() and (wide[:, 16 + w:] == 3.0).all()


def test_linear_zero_state_and_out_of_place(eng):
    for new in ([1, 2], [100, 30]):
        c = LinearCase(new, 1, 2, 64, 128, torch.bfloat16, seed=23)
        s0 = c.state.to(DEV)
        so = torch.full_like(s0, 9.0)
        out, state = c.run(eng, state=s0, state_out=so)
        assert state is so and torch.equal(s0.cpu(), c.state)
        c.check(out, state)
        so2 = torch.full_like(s0, 9.0)
        out, state = eng.linattn(c.gq, c.gk, c.gv, c.gg, c.start, None, state_out=so2, slots=c.slots.to(DEV),
                                 max_new=max(new))
        c.check(out, state, zero=True)
        unused = (set(range(3)) - set(c.slots.tolist())).pop()
        assert (so2[unused] == 9.0).all()
    assert eng.sync_status() == q4.Q4_OK


def test_linear_in_pieces_is_the_whole(eng):
    """A prompt in chunks, then token by token, ends in the state of one pass."""
    c = LinearCase([200], 1, 2, 128, 128, torch.float16, seed=24, slots=torch.tensor([0], dtype=torch.int32))
    whole, end = c.run(eng)
    c.check(whole, end)
    state = c.state.to(DEV)
    parts = []
    for a, b in [(0, 90), (90, 91), (91, 190)] + [(i, i + 1) for i in range(190, 200)]:
        o, _ = eng.linattn(c.gq[a:b], c.gk[a:b], c.gv[a:b], c.gg[a:b], ints([0, b - a]), state, max_new=b - a)
        parts.append(o)
    assert eng.sync_status() == q4.Q4_OK
    c.check(torch.cat(parts), state)


def test_linear_bad_slots_are_left_out(eng):
    for new in ([1, 1, 1], [70, 80, 90]):
        c = LinearCase(new, 1, 1, 64, 64, torch.float16, seed=25)
        bad = c.slots.clone()
        bad[1] = 99
        out0 = torch.full((c.rows, 1, 64), 3.0, dtype=torch.float16, device=DEV)
        out, state = c.run(eng, slots=bad.to(DEV), out=out0)
        assert eng.sync_status() == q4.Q4_EINDEX
        at = starts(new)
        assert (out[at[1]:at[2]] == 3.0).all()
        assert torch.equal(state[c.slots[1]].cpu(), c.state[c.slots[1]])
        c.check(out, state, seqs=[0, 2])


def test_linear_rows_of_no_sequence_and_graph(eng):
    for new in ([1, 1], [100, 65]):
        c = LinearCase(new, 1, 2, 64, 64, torch.float16, seed=26)
        q, k, v = (torch.cat((x, torch.full_like(x[:2], float("nan")))) for x in (c.gq, c.gk, c.gv))
        g = torch.cat((c.gg, c.gg[:2]))
        out = torch.full((c.rows + 2, 2, 64), 3.0, dtype=torch.float16, device=DEV)
        so = torch.zeros(3, 2, 64, 64, device=DEV)
        s0, slots = c.state.to(DEV), c.slots.to(DEV)
        call = lambda: eng.linattn(q, k, v, g, c.start, s0, state_out=so, slots=slots, out=out, max_new=max(new))  # noqa: E731
        call()
        assert eng.sync_status() == q4.Q4_OK
        c.check(out[:c.rows], so)
        assert (out[c.rows:] == 3.0).all()
        first, fs = out.clone(), so.clone()
        out.fill_(0)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        gr.replay()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:c.rows], first[:c.rows]) and torch.equal(so, fs)


# ---- refusals ---------------------------------------------------------------

def test_refusals(eng):
    c = AttendCase([2], [40], 4, 2, 64, 16, torch.float16, seed=30)
    f = eng.rope_freqs(64)
    q3 = c.gq

    def refuses(status, call):
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == status, e.value

    ap = lambda **kw: eng.attn_paged(c.cache, c.start, c.glen, kw.pop("q", q3), **kw)  # noqa: E731
    refuses(q4.Q4_EINVAL, lambda: ap(out=q3))
    refuses(q4.Q4_EINVAL, lambda: ap(window=-1))
    refuses(q4.Q4_EINVAL, lambda: ap(max_new=0))
    refuses(q4.Q4_EINVAL, lambda: ap(scale=float("nan")))
    refuses(q4.Q4_EINVAL, lambda: ap(q=q3.float()))
    refuses(q4.Q4_EINVAL, lambda: ap(q=q3.bfloat16()))
    refuses(q4.Q4_EINVAL, lambda: ap(q=q3.cpu()))
    refuses(q4.Q4_ESHAPE, lambda: ap(q=q3[:, :3].contiguous()))
    refuses(q4.Q4_ESHAPE, lambda: ap(q=q3[..., :32]))
    refuses(q4.Q4_ESHAPE, lambda: ap(out=torch.empty(3, 4, 64, dtype=torch.float16, device=DEV)))
    refuses(q4.Q4_EALIGN, lambda: ap(q=torch.zeros(2 * 256 + 8, dtype=torch.float16, device=DEV)[1:513].view(2, 4, 64)))
    refuses(q4.Q4_ESHAPE, lambda: ap(q=torch.zeros(2, 260, dtype=torch.float16, device=DEV)[:, :256].unflatten(1, (4, 64))))
    refuses(q4.Q4_ESHAPE, lambda: eng.attn_paged(c.cache, c.start[:1], c.glen, q3))
    refuses(q4.Q4_EINVAL, lambda: eng.attn_paged(c.cache, c.start.long(), c.glen, q3))
    refuses(q4.Q4_ESHAPE, lambda: eng.attn_paged(c.cache, ints([0, 1, 2]), ints([1, 1]), q3))

    k, v = c.cache.k, c.cache.v
    refuses(q4.Q4_ESHAPE, lambda: q4.PagedKV(k, v[:, :8], c.cache.table))
    refuses(q4.Q4_EINVAL, lambda: q4.PagedKV(k.float(), v.float(), c.cache.table))
    refuses(q4.Q4_ESHAPE, lambda: q4.PagedKV(k, v, c.cache.table.long()))
    refuses(q4.Q4_ESHAPE, lambda: q4.PagedKV(k.transpose(2, 3), v.transpose(2, 3), c.cache.table))
    odd = torch.zeros(4, 16, 2, 20, dtype=torch.float16, device=DEV)
    refuses(q4.Q4_ESHAPE, lambda: eng.attn_paged(q4.PagedKV(odd, odd.clone(), c.cache.table), c.start, c.glen,
                                                 torch.zeros(2, 4, 20, dtype=torch.float16, device=DEV)))

    nk = torch.zeros(2, 2, 64, dtype=torch.float16, device=DEV)
    apd = lambda **kw: eng.kv_append(c.cache, c.start, c.glen, kw.pop("k", nk), kw.pop("v", nk), **kw)  # noqa: E731
    refuses(q4.Q4_ESHAPE, lambda: apd(freqs=eng.rope_freqs(128)))
    refuses(q4.Q4_EINVAL, lambda: apd(freqs=f.float()))
    refuses(q4.Q4_EINVAL, lambda: apd(freqs=f, amp=float("inf")))
    refuses(q4.Q4_ESHAPE, lambda: apd(v=nk[:1]))
    refuses(q4.Q4_ESHAPE, lambda: apd(k=nk[:, :1]))
    refuses(q4.Q4_ESHAPE, lambda: apd(pos=ints([1])))
    refuses(q4.Q4_EINVAL, lambda: apd(q=q3, q_out=q3.bfloat16()))

    lc = LinearCase([2], 1, 2, 64, 64, torch.float16, seed=31)
    s = lc.state.to(DEV)
    la = lambda **kw: eng.linattn(kw.pop("q", lc.gq), kw.pop("k", lc.gk), kw.pop("v", lc.gv),  # noqa: E731
                                  kw.pop("g", lc.gg), lc.start, kw.pop("state", s), **kw)
    refuses(q4.Q4_EINVAL, lambda: la(state=None))
    refuses(q4.Q4_ESHAPE, lambda: la(state=s[:, :1]))
    refuses(q4.Q4_ESHAPE, lambda: la(state=s.half()))
    refuses(q4.Q4_ESHAPE, lambda: la(state_out=s.transpose(2, 3)))
    refuses(q4.Q4_ESHAPE, lambda: la(g=lc.gg.half()))
    refuses(q4.Q4_ESHAPE, lambda: la(g=lc.gg[:, :1]))
    refuses(q4.Q4_EINVAL, lambda: la(k=lc.gk.bfloat16()))
    refuses(q4.Q4_ESHAPE, lambda: la(k=lc.gk[:1]))
    refuses(q4.Q4_EINVAL, lambda: la(scale=float("inf")))
    refuses(q4.Q4_EINVAL, lambda: la(max_new=0))
    refuses(q4.Q4_EINVAL, lambda: la(out=lc.gv))
    refuses(q4.Q4_ESHAPE, lambda: la(slots=ints([0, 1])))
    refuses(q4.Q4_ESHAPE, lambda: eng.linattn(lc.gq, lc.gk, lc.gv, lc.gg, ints([0, 1, 2]), s[:1]))
    assert eng.sync_status() == q4.Q4_OK


def test_fault_injection_reaches_these_calls(eng):
    c = AttendCase([1], [20], 2, 1, 64, 16, torch.float16, seed=32)
    lc = LinearCase([1], 1, 1, 64, 64, torch.float16, seed=32)
    eng.set_fault("launch")
    try:
        for call in (lambda: c.run(eng), lambda: lc.run(eng),
                     lambda: eng.kv_append(c.cache, c.start, c.glen, c.gq[:, :1], c.gq[:, 1:])):
            with pytest.raises(q4.Q4Error) as e:
                call()
            assert e.value.status == q4.Q4_EFAULTINJ
    finally:
        eng.set_fault("none")
    c.check(c.run(eng))


def test_empty_batches(eng):
    c = AttendCase([1], [20], 2, 1, 64, 16, torch.float16, seed=33)
    none = c.gq[:0]
    assert eng.attn_paged(c.cache, ints([0, 0]), ints([5]), none).shape == (0, 2, 64)
    assert eng.attn_paged(c.cache, ints([0]), ints([]), none).shape == (0, 2, 64)
    eng.kv_append(c.cache, ints([0, 0]), ints([5]), none[:, :1], none[:, :1])
    lc = LinearCase([1], 1, 1, 64, 64, torch.float16, seed=33)
    s0 = lc.state.to(DEV)
    so = torch.zeros_like(s0)
    out, _ = eng.linattn(lc.gq[:0], lc.gk[:0], lc.gv[:0], lc.gg[:0], ints([0, 0]), s0, state_out=so)
    assert out.shape == (0, 1, 64)
    assert torch.equal(so[0], s0[0]) and (so[1] == 0).all()      # a sequence without tokens copies its state
    assert eng.sync_status() == q4.Q4_OK


def test_streams(eng):
    """Inputs made on one stream, the calls on another, the default left alone."""
    side = torch.cuda.Stream()
    c = AttendCase([1, 40], [200, 60], 4, 2, 128, 16, torch.float16, seed=34)
    side.wait_stream(torch.cuda.current_stream())
    out = c.run(eng, max_new=40, stream=side)
    out2 = c.run(eng, max_new=40, stream=side.cuda_stream)
    assert eng.sync_status(side) == q4.Q4_OK
    c.check(out)
    assert torch.equal(out, out2)


def test_first_calls_of_a_process_in_a_capture():
    """A process whose first launch of each kernel is in a graph's capture."""
    code = """
import torch, q4_quantized_decode_b200 as q4
d = "cuda:0"
eng = q4.Q4Gemv(0)
gen = torch.Generator().manual_seed(1)
t = lambda *s: torch.randn(*s, generator=gen).half().to(d)
i = lambda *x: torch.tensor(x, dtype=torch.int32, device=d)
f = eng.rope_freqs(64)
q, k, v, g = t(140, 4, 64), t(140, 2, 64), t(140, 2, 64), -torch.rand(140, 2, generator=gen).to(d)
table, start, length = i(*range(9)).view(1, 9), i(0, 140), i(140)

def run(cache, state):
    rq = eng.kv_append(cache, start, length, k, v, q=q, freqs=f)
    o = eng.attn_paged(cache, start, length, rq, max_new=140)
    a, _ = eng.linattn(k, k, v, g, start, state, max_new=1)
    b, _ = eng.linattn(k, k, v, g, start, state, max_new=2000)
    return o, a, b, cache.k, state

def fresh():
    z = torch.zeros(9, 16, 2, 64, dtype=torch.float16, device=d)
    return q4.PagedKV(z, z.clone(), table), torch.zeros(1, 2, 64, 64, device=d)

x = fresh()
s = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(s):
    got = run(*x)
s.replay()
torch.cuda.synchronize()
want = run(*fresh())
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert eng.sync_status() == q4.Q4_OK
del s
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


# ---- a run of them together -------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_then_tokens(eng, dtype):
    """A prompt in two ragged chunks, then tokens one at a time: append and
    attend on one cache give what attention over the whole sequence gives."""
    hq, hkv, dim, page = 4, 2, 64, 16
    total = [90, 41]
    steps = [[70, 30], [15, 9], [1, 1], [1, 0], [1, 1], [2, 0]]
    gen = torch.Generator().manual_seed(40)
    table, pool = ref.table_of(total, page, gen)
    nan = lambda: torch.full((pool, page, hkv, dim), float("nan"), dtype=dtype, device=DEV)  # noqa: E731
    cache = q4.PagedKV(nan(), nan(), table.to(DEV))
    x = [torch.randn(t, (hq + 2 * hkv), dim, generator=gen).to(dtype) for t in total]
    freqs = eng.rope_freqs(dim // 2, base=500.0)
    done, outs = [0, 0], [[], []]
    for new in steps:
        rows = torch.cat([x[s][done[s]:done[s] + n] for s, n in enumerate(new)]).to(DEV)
        done = [d + n for d, n in zip(done, new)]
        start, length = ints(starts(new)), ints(done)
        q = eng.kv_append(cache, start, length, rows[:, hq:hq + hkv], rows[:, hq + hkv:], q=rows[:, :hq], freqs=freqs)
        o = eng.attn_paged(cache, start, length, q, max_new=max(new))
        outs[0].append(o[:new[0]])
        outs[1].append(o[new[0]:])
    assert eng.sync_status() == q4.Q4_OK and done == total
    u = ref.half_step(dtype)
    for s, t in enumerate(total):
        pos = torch.arange(t)
        got = torch.cat(outs[s])
        q, _ = ref.rotate(x[s][:, :hq], pos, freqs.cpu())
        k, _ = ref.rotate(x[s][:, hq:hq + hkv], pos, freqs.cpu())
        q, k = q.to(dtype), k.to(dtype)                  # as stored
        for h in range(hq):
            v = x[s][:, hq + hkv + h // 2]
            o, a, mags = ref.attend(q[:, h], k[:, h // 2], v, 0, dim ** -0.5)
            # a stored value off by one rounding the other way moves a score by 2 u mags
            tol = (u + (2 * dim * 2.0 ** -23 + 8 * u) * mags[:, None] + 2.0 ** -18) * a + t * 2.0 ** -25 * 6 + \
                u * o.abs() + ref.tiny(dtype)
            close(got[:, h], o, tol, f"sequence {s}, head {h}")
