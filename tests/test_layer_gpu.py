"""The draft layer's attention on the GPU against the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
  rotated value   3 roundings over |a| + |b|: 4 u (|a| + |b|)
  scale           4 u * 2 relative (a pair's |a| + |b| is at most 2 amax), and one division: 16 u
  code            within 0.5 of the float64 value, and 128 * 32 u for the value's own error: 0.5 + 2^-12
  q out           bf16's half ulp (of 8 significant bits) at the value, and the rotation's error
  read            bit for bit: one product and one rounding
  z               D products summed in fp32: D u sum |q||k|; two more operations on z and the running maximum: 8 u |z|
  lse             z's error and 2^-20 for the logarithms and sums of positive terms
  out             weights rounded to 11 bits (2^-11) and perturbed by z's error: (2^-11 + 2 dz + 2^-18) sum p|v|, then bf16's half ulp
"""
import numpy as np
import pytest

from bit_quantized_lm_amd import _binding as B
from bit_quantized_lm_amd import _layer as L
from oracle import layer as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    B.load_library()
    return torch.device("cuda:0")


def half_ulp(x):
    """Half a bf16 ulp at x, with room for a neighbour one binade up."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -120) * (1 + 2.0 ** -8))) - 8)


def bf16(rng, *shape, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16)


class Case:
    """A cache with random contents and a batch over it, on the host and the GPU."""

    def __init__(self, dev, lens, hq, hkv, d, page, seed, spare=3, max_pages=None):
        rng = self.rng = np.random.default_rng(seed)
        self.dev, self.lens, self.hq, self.hkv, self.d, self.page = dev, lens, hq, hkv, d, page
        need = [max(0, -(-l // page)) for _, l in lens]
        self.max_pages = max_pages or max(1, max(need)) + 1
        n_pages = self.n_pages = sum(need) + spare
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(lens), self.max_pages), -7, np.int32)     # unused entries are no page at all
        at = 0
        for s, n in enumerate(need):
            n = min(n, self.max_pages)
            self.table[s, :n] = order[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([l for _, l in lens], np.int32)
        self.rows = int(self.q_start[-1])
        shape = (n_pages, hkv, page, d)
        self.kc = np.clip(np.rint(rng.standard_normal(shape) * 33), -127, 127).astype(np.int16) + 128
        self.vc = np.clip(np.rint(rng.standard_normal(shape) * 33), -127, 127).astype(np.int16) + 128
        self.kc, self.vc = self.kc.astype(np.uint8), self.vc.astype(np.uint8)
        self.ks = rng.uniform(0.01, 0.06, shape[:2]).astype(np.float32)
        self.vs = rng.uniform(0.01, 0.06, shape[:2]).astype(np.float32)
        self.q = bf16(rng, self.rows, hq, d)

    def upload(self):
        to = lambda a: torch.from_numpy(a).to(self.dev)  # noqa: E731
        self.cache = [to(a) for a in (self.kc, self.vc, self.ks, self.vs)]
        self.batch = [to(a) for a in (self.q_start, self.kv_len, self.table)]
        return self

    def naturals(self):
        return O.natural(self.kc, O.key_byte), O.natural(self.vc, O.value_byte)


# ------------------------------------------------------------------- append
APPENDS = [
    # lens [(new, in cache)], hq, hkv, d, page, rot, interleaved
    ([(1, 1)], 2, 1, 64, 32, 64, False),
    ([(1, 778)], 40, 8, 128, 64, 128, False),
    ([(1, 64), (1, 65), (1, 128)], 5, 1, 128, 64, 128, True),
    ([(9, 70), (0, 40), (9, 9), (3, 131)], 8, 2, 128, 64, 64, True),
    ([(200, 200)], 4, 4, 64, 32, 32, False),
    ([(67, 167), (33, 33)], 6, 3, 256, 256, 256, False),
    ([(300, 555)], 3, 3, 256, 128, 16, True),
    ([(31, 95), (1, 32), (32, 64)], 7, 7, 64, 32, 0, False),
    ([(5, 3), (2, 0)], 4, 2, 64, 32, 64, False),                   # rows of negative positions
    ([(1, i + 1) for i in range(130)], 2, 2, 64, 32, 64, False),   # more sequences than a wave has lanes
]


def check_append(c, got_q, rope, interleaved, k, v, before, with_q=True):
    kn, vn = before
    q_want, pages = O.append(c.q.float().numpy() if with_q else None, k.float().numpy(), v.float().numpy(),
                             rope, kn, vn, c.ks, c.vs, c.q_start, c.kv_len, c.table, interleaved)
    if with_q:
        q = c.q.double().numpy()
        slack = 8 * U * np.abs(q).max(axis=2, keepdims=True)
        assert np.all(np.abs(got_q.double().cpu().numpy() - q_want) <= half_ulp(q_want) + slack)
    kc, vc, ks, vs = (t.cpu().numpy() for t in c.cache)
    for w, (codes, scale, was, byte_of, old_scale) in enumerate(((kc, ks, kn, O.key_byte, c.ks), (vc, vs, vn, O.value_byte, c.vs))):
        now = O.natural(codes, byte_of)
        assert now.min() >= -127
        for pid in range(c.n_pages):
            for h in range(c.hkv):
                p = pages.get((pid, h, w))
                if p is None:
                    assert scale[pid, h] == old_scale[pid, h] and np.array_equal(now[pid, h], was[pid, h])
                    continue
                assert abs(scale[pid, h] - p["step"]) <= 16 * U * p["step"], (pid, h, w)
                for t in range(c.page):
                    if t not in p["want"]:
                        assert np.array_equal(now[pid, h, t], was[pid, h, t]), (pid, h, w, t)
                    elif t in p["old"] and p["kept"]:
                        assert np.array_equal(now[pid, h, t], was[pid, h, t]), (pid, h, w, t)
                    else:
                        assert np.abs(now[pid, h, t] - p["want"][t]).max() <= 0.5 + 2.0 ** -12, (pid, h, w, t)


@pytest.mark.parametrize("lens,hq,hkv,d,page,rot,interleaved", APPENDS)
def test_append(dev, lens, hq, hkv, d, page, rot, interleaved):
    c = Case(dev, lens, hq, hkv, d, page, seed=rot + d + len(lens)).upload()
    before = c.naturals()
    rope = L.draft_layer_rope_table(c.max_pages * page, rot) if rot else None
    # values that raise some scales and not others; q, k and v are slices of one projection
    k, v = bf16(c.rng, c.rows, hkv, d, scale=1.2), bf16(c.rng, c.rows, hkv, d, scale=1.2)
    qkv = torch.cat([c.q, k, v], dim=1).to(dev)
    q, kk, vv = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    got = L.draft_layer_append(q, kk, vv, None if rope is None else torch.from_numpy(rope).to(dev), *c.cache, *c.batch,
                               interleaved=interleaved)
    torch.cuda.synchronize()
    check_append(c, got, rope, interleaved, k, v, before)
    # the same call again leaves the same bytes
    first = [t.clone() for t in c.cache]
    again = L.draft_layer_append(q, kk, vv, None if rope is None else torch.from_numpy(rope).to(dev), *c.cache, *c.batch,
                                 interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(got, again) and all(torch.equal(a, b) for a, b in zip(first, c.cache))


def test_append_without_queries_and_in_place(dev):
    c = Case(dev, [(6, 70), (2, 2)], 4, 2, 128, 64, seed=5).upload()
    before = c.naturals()
    rope = L.draft_layer_rope_table(c.max_pages * 64, 128)
    k, v = bf16(c.rng, c.rows, 2, 128), bf16(c.rng, c.rows, 2, 128)
    t = torch.from_numpy(rope).to(dev)
    assert L.draft_layer_append(None, k.to(dev), v.to(dev), t, *c.cache, *c.batch) is None
    torch.cuda.synchronize()
    check_append(c, None, rope, False, k, v, before, with_q=False)
    q = c.q.to(dev)
    apart = L.draft_layer_append(q, k.to(dev), v.to(dev), t, *c.cache, *c.batch)
    here = q.clone()
    assert L.draft_layer_append(here, k.to(dev), v.to(dev), t, *c.cache, *c.batch, q_out=here) is here
    assert torch.equal(here, apart)


def test_append_zero_values_and_stale_scale(dev):
    """A page that starts afresh takes no part of what it held (a NaN scale
    included); zeros get the smallest scale; an old scale stays where it is the larger."""
    c = Case(dev, [(3, 3), (2, 34)], 1, 1, 64, 32, seed=6)
    c.ks[c.table[0, 0]] = np.nan
    c.vs[c.table[0, 0]] = np.inf
    c.ks[c.table[1, 1]] = np.nan
    c.upload()
    k = torch.zeros((c.rows, 1, 64), dtype=torch.bfloat16)
    v = bf16(c.rng, c.rows, 1, 64)
    L.draft_layer_append(None, k.to(dev), v.to(dev), None, *c.cache, *c.batch)
    torch.cuda.synchronize()
    ks, vs = c.cache[2].cpu().numpy(), c.cache[3].cpu().numpy()
    assert ks[c.table[0, 0], 0] == 2.0 ** -40 and ks[c.table[1, 1], 0] == 2.0 ** -40
    assert vs[c.table[0, 0], 0] == np.float32(v[:3].float().abs().max().item()) / np.float32(127)
    got = O.natural(c.cache[0].cpu().numpy(), O.key_byte)
    assert np.all(got[c.table[0, 0], 0, :3] == 0)


def test_append_token_by_token_stays_near(dev):
    """A page filled one token at a time, its scale rising as larger tokens come:
    each rise re-rounds the older codes once more (half a step each)."""
    d, page, n = 64, 32, 32
    c = Case(dev, [(1, n)], 1, 1, d, page, seed=7).upload()
    rng = c.rng
    v = bf16(rng, n, 1, d) * torch.linspace(0.3, 3.0, n)[:, None, None].to(torch.bfloat16)
    scales = []
    for i in range(n):
        c.batch[1].fill_(i + 1)
        L.draft_layer_append(None, v[i:i + 1].to(dev), v[i:i + 1].to(dev), None, *c.cache, *c.batch)
        scales.append(c.cache[3].cpu().numpy()[c.table[0, 0], 0])
    assert scales == sorted(scales)
    _, got = L.draft_layer_read(*c.cache, torch.tensor([0, n], dtype=torch.int32, device=dev), c.batch[1], c.batch[2], n)
    want = v.float().numpy()
    bound = np.array([0.5 * s + 0.5 * sum(b for a, b in zip(scales[i:], scales[i + 1:]) if b > a) for i, s in enumerate(scales)])
    assert np.all(np.abs(got.float().cpu().numpy() - want).max(axis=(1, 2)) <= bound * (1 + 2.0 ** -7) + half_ulp(np.abs(want).max(axis=(1, 2))))


def test_bad_pages_are_left_alone(dev):
    """Tokens whose page id is outside the pool are not written, read as zero
    and not seen."""
    c = Case(dev, [(40, 100)], 2, 1, 64, 32, seed=8)
    c.table[0, 2] = c.n_pages
    c.upload()
    before = c.naturals()
    k, v = bf16(c.rng, c.rows, 1, 64), bf16(c.rng, c.rows, 1, 64)
    got = L.draft_layer_append(c.q.to(dev), k.to(dev), v.to(dev), None, *c.cache, *c.batch)
    torch.cuda.synchronize()
    check_append(c, got, None, False, k, v, before)
    kb, vb = L.draft_layer_read(*c.cache, *c.batch, c.rows)
    pos = np.arange(60, 100)
    assert not kb.cpu()[(pos >= 64) & (pos < 96)].any() and not vb.cpu()[(pos >= 64) & (pos < 96)].any()
    assert kb.cpu()[pos < 64].any()
    c.kc, c.vc, c.ks, c.vs = (t.cpu().numpy() for t in c.cache)
    check_attend(c, window=0, sinks=0)


@pytest.mark.parametrize("new", [1, 40])
def test_missing_page_takes_nothing_from_page_zero(dev, new):
    """A page that is not there is hidden whatever the pool's first page holds."""
    c = Case(dev, [(new, 200)], 4, 1, 64, 32, seed=21, spare=4)
    used = c.table[0, :7].copy()
    other = next(p for p in range(c.n_pages) if p not in used and p != 0)
    c.table[0, :7] = np.where(used == 0, other, used)     # page 0 is nobody's
    c.table[0, 3] = -1
    c.ks[0], c.vs[0], c.kc[0], c.vc[0] = np.inf, np.inf, 255, 255
    c.upload()
    check_attend(c, 0, 0)
    c.ks[0], c.vs[0] = np.nan, np.nan
    c.upload()
    check_attend(c, 0, 0)


def test_past_the_tables_end(dev):
    """Positions that the table has no entry for are not written, read as zero and not seen."""
    c = Case(dev, [(40, 100), (2, 300)], 2, 1, 64, 32, seed=22, max_pages=2).upload()
    before = c.naturals()
    rope = L.draft_layer_rope_table(64, 64)
    k, v = bf16(c.rng, c.rows, 1, 64), bf16(c.rng, c.rows, 1, 64)
    got = L.draft_layer_append(c.q.to(dev), k.to(dev), v.to(dev), torch.from_numpy(rope).to(dev), *c.cache, *c.batch)
    torch.cuda.synchronize()
    check_append(c, got, rope, False, k, v, before)
    kb, vb = L.draft_layer_read(*c.cache, *c.batch, c.rows)
    assert kb.cpu()[:4].any() and not kb.cpu()[4:].any() and not vb.cpu()[4:].any()
    c.kc, c.vc, c.ks, c.vs = (t.cpu().numpy() for t in c.cache)
    for window, sinks in ((0, 0), (50, 3)):
        check_attend(c, window, sinks)


@pytest.mark.parametrize("hkv,new", [(1, 20), (8, 20), (8, 3), (2, 40)])
def test_attend_many_sequences(dev, hkv, new):
    """More sequences than a wave has lanes, in each way that tiles become workgroups."""
    lens = [(new + i % 5 if i % 9 else 0, 60 + (37 * i) % 400) for i in range(70)]
    check_attend(Case(dev, lens, hkv * 2, hkv, 64, 32, seed=hkv + new).upload(), 0, 0)


@pytest.mark.parametrize("new,d,hkv,window", [(1, 64, 8, 0), (9, 64, 8, 0), (1, 128, 8, 700), (70, 64, 4, 0)])
def test_attend_uneven_lengths(dev, new, d, hkv, window):
    """Thirty tiles a head of lengths far apart: runs that hold the end of one tile and the start of another."""
    lens = [(new, new + 5 + 200 * i) for i in range(30)]
    check_attend(Case(dev, lens, hkv * 2, hkv, d, 64, seed=new + d).upload(), window, 4 if window else 0)


# --------------------------------------------------------------------- read
@pytest.mark.parametrize("lens,hkv,d,page", [
    ([(1, 1)], 1, 64, 32), ([(500, 500)], 8, 128, 64), ([(33, 97), (0, 5), (64, 64), (1, 300)], 5, 128, 128),
    ([(77, 500), (256, 256)], 3, 256, 256), ([(5, 3), (3, 0)], 2, 64, 32), ([(1, i + 1) for i in range(70)], 1, 64, 32)])
def test_read(dev, lens, hkv, d, page):
    c = Case(dev, lens, hkv, hkv, d, page, seed=page + d).upload()
    kb, vb = L.draft_layer_read(*c.cache, *c.batch, c.rows)
    torch.cuda.synchronize()
    kn, vn = c.naturals()
    for got, n, scale in ((kb, kn, c.ks), (vb, vn, c.vs)):
        want = np.zeros((c.rows, hkv, d), np.float32)
        for s, r, p in O.positions_of(c.q_start, c.kv_len):
            if p >= 0:
                pid = c.table[s, p // page]
                want[r] = n[pid, :, p % page].astype(np.float32) * scale[pid][:, None]
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


# ------------------------------------------------------------------- attend
def check_attend(c, window, sinks, q=None, scale=None, **kw):
    qd = c.q.to(c.dev) if q is None else q
    scale = 1.0 / np.sqrt(c.d) if scale is None else scale
    out, lse = L.draft_layer_attend(qd, *c.cache, *c.batch, scale=scale, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    kn, vn = c.naturals()
    want, lwant, spread, absqk = O.attend(c.q.float().numpy(), kn, vn, c.ks, c.vs, c.q_start, c.kv_len, c.table, scale, window, sinks)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    dz = (c.d + 16) * U * absqk
    none = np.isneginf(lwant)
    assert np.array_equal(np.isneginf(lse), none) and not np.isnan(lse).any()
    assert np.all(np.abs(lse - lwant)[~none] <= (dz + 2.0 ** -20 + 4 * U * np.abs(lwant))[~none])
    err, lim = np.abs(out - want), half_ulp(want) + (2.0 ** -11 + 2 * dz[..., None] + 2.0 ** -18) * spread
    assert np.all(err <= lim), (err - lim).max()
    assert not out[none].any()
    return out, lse


ATTENDS = [
    # lens, hq, hkv, d, page, window, sinks
    ([(1, 1)], 1, 1, 64, 32, 0, 0),
    ([(1, 33)], 5, 1, 128, 64, 0, 0),
    ([(1, 1000)], 40, 8, 128, 64, 0, 0),
    ([(1, 20011)], 8, 1, 64, 128, 0, 0),                                   # one row split over the card
    ([(1, 3000)], 16, 2, 256, 256, 0, 0),
    ([(9, 700), (9, 9), (0, 50), (4, 1290)], 10, 2, 128, 64, 0, 0),
    ([(3, 517), (1, 2), (2, 4000)], 21, 3, 64, 32, 0, 0),                  # heads and groups of odd numbers
    ([(130, 130)], 2, 2, 128, 64, 0, 0),
    ([(77, 300), (250, 250)], 12, 3, 128, 32, 0, 0),
    ([(100, 400), (65, 65)], 8, 1, 256, 128, 0, 0),
    ([(600, 1111)], 2, 1, 64, 64, 0, 0),
    ([(1, 1000), (1, 10)], 4, 2, 64, 32, 100, 4),
    ([(9, 1000), (9, 20)], 5, 1, 128, 64, 64, 0),
    ([(40, 777)], 6, 2, 128, 64, 1, 0),                                    # a row sees itself alone
    ([(40, 777)], 6, 2, 128, 64, 1, 3),
    ([(300, 900)], 4, 2, 128, 128, 200, 70),                               # sinks over several groups
    ([(200, 500)], 3, 1, 256, 64, 33, 1),
    ([(50, 400)], 2, 2, 64, 32, 100000, 4),                                # a window past everything
    ([(90, 90)], 2, 2, 64, 32, 7, 500),                                    # sinks past everything
    ([(5, 3), (3, 0), (2, 2)], 4, 2, 64, 32, 0, 0),                        # rows that see nothing
    ([(40, 20)], 8, 2, 128, 64, 8, 2),
    ([(1, 5 + 7 * i) for i in range(150)], 4, 1, 64, 32, 0, 0),            # more sequences than a wave has lanes
    ([(1, 9000)] + [(1, 3)] * 20, 8, 2, 128, 64, 0, 0),                    # lengths far apart
]


@pytest.mark.parametrize("lens,hq,hkv,d,page,window,sinks", ATTENDS)
def test_attend(dev, lens, hq, hkv, d, page, window, sinks):
    c = Case(dev, lens, hq, hkv, d, page, seed=hq * 1000 + d + len(lens)).upload()
    check_attend(c, window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 2, 3, 4, 7, 8, 13, 16, 30, 33, 64, 65, 128, 129, 257])
def test_attend_row_counts(dev, d, new):
    """Every tile height, on both sides of its edges."""
    c = Case(dev, [(new, new + 75)], 5, 1, d, 64, seed=new).upload()
    check_attend(c, 0, 0)


def test_attend_hidden_contents_do_not_matter(dev):
    """What a row does not see (later tokens' codes, scales of NaN and infinity
    on pages and tokens past the length or before the window) changes nothing."""
    c = Case(dev, [(4, 300), (1, 70)], 4, 2, 64, 32, seed=11, max_pages=12)
    spare = [p for p in range(c.n_pages) if p not in c.table]
    c.table[0, 10:] = spare[:2]                        # pages past the length, in the table
    a = c.upload()
    first = check_attend(a, window=40, sinks=4)
    seen = set(c.table[0, [0, 8, 9]]) | set(c.table[1, [0, 1, 2]])
    for p in range(c.n_pages):
        if p not in seen:
            c.ks[p], c.vs[p] = np.nan, np.inf
            c.kc[p], c.vc[p] = 255, 255
    for codes, byte_of in ((c.kc, O.key_byte), (c.vc, O.value_byte)):      # tokens past the length on the last pages
        t, e = np.meshgrid(np.arange(300 - 288, 32), np.arange(64), indexing="ij")
        codes[c.table[0, 9]].reshape(2, -1)[:, byte_of(t, e, 64)] = 0
    second = c.upload()
    out, lse = L.draft_layer_attend(c.q.to(dev), *second.cache, *second.batch, window=40, sinks=4)
    assert np.array_equal(out.double().cpu().numpy(), first[0]) and np.array_equal(lse.double().cpu().numpy(), first[1])


def test_attend_extreme_scores(dev):
    """Rows whose scores spread over hundreds (one token takes all), a row of
    zeros, rows of tiny and of huge elements, and page scales far apart."""
    c = Case(dev, [(6, 500)], 2, 1, 128, 64, seed=12)
    x = c.q.float()
    x[0] *= 60.0
    x[1] = 0.0
    x[2] *= 1e-20
    x[3, :, 5] = 3.0e4
    x[4] *= 2.0 ** -60
    c.q = x.to(torch.bfloat16)
    c.vs[c.table[0, 2]] = 2.0 ** -40
    c.vs[c.table[0, 3]] = 2.0 ** 20
    c.ks[c.table[0, 4]] = 0.0
    c.upload()
    check_attend(c, 0, 0)


def test_attend_many_small_weights(dev):
    """One token outweighs each of 20,000 others by 2^12, which together outweigh
    it: their weights must keep their share."""
    d, n = 64, 20000
    c = Case(dev, [(1, n)], 1, 1, d, 64, seed=13)
    c.kc[:] = 128
    t, e = np.meshgrid(np.array([0]), np.arange(d), indexing="ij")
    c.kc[c.table[0, 0], 0].reshape(-1)[O.key_byte(t, e, d)] = 128 + 64
    c.ks[:] = 1.0 / 64
    c.q = torch.full((1, 1, d), 0.13, dtype=torch.float32).to(torch.bfloat16)
    c.upload()
    check_attend(c, 0, 0, scale=1.0)


def test_attend_nan_row_stays_alone(dev):
    c = Case(dev, [(9, 200)], 5, 1, 64, 32, seed=14).upload()
    out, lse = check_attend(c, 0, 0)
    q = c.q.clone()
    q[3, 2, 7] = float("nan")
    q[5, 1, 0] = float("inf")
    got, glse = L.draft_layer_attend(q.to(dev), *c.cache, *c.batch)
    got, glse = got.double().cpu().numpy(), glse.double().cpu().numpy()
    bad = np.zeros((9, 5), bool)
    bad[3, 2] = bad[5, 1] = True
    assert np.isnan(got[bad]).any(axis=1).all()
    assert np.array_equal(got[~bad], out[~bad]) and np.array_equal(glse[~bad], lse[~bad])


def test_attend_strided_queries_given_outputs_and_repeats(dev):
    """Queries inside a wider row; the caller's own outputs; a workspace that
    serves calls of other sizes; every repeat gives the same bits."""
    c = Case(dev, [(2, 5000), (1, 9000)], 8, 2, 64, 64, seed=15).upload()
    wide = torch.full((c.rows, 12, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 2:10] = c.q.to(dev)
    ws = L.draft_layer_workspace(4000, 1, 8, 2, 256, dev)
    out = torch.empty((c.rows, 8, 64), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((c.rows, 8), dtype=torch.float32, device=dev)
    first = check_attend(c, 0, 0, q=wide[:, 2:10], out=out, lse=lse, workspace=ws)
    other = Case(dev, [(70, 3000), (1, 8000)], 16, 2, 256, 128, seed=16).upload()
    for _ in range(3):
        check_attend(other, 0, 0, workspace=ws)
        again = check_attend(c, 0, 0, workspace=ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_other_stream(dev):
    """Calls on a stream of their own, outputs allocated by the binding."""
    c = Case(dev, [(9, 3000), (9, 100)], 8, 2, 128, 64, seed=17).upload()
    want = L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch)
    q = c.q.to(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = L.draft_layer_attend(q, *c.cache, *c.batch, stream=s)
    kb, vb = L.draft_layer_read(*c.cache, *c.batch, c.rows, stream=s.cuda_stream)
    junk = [torch.full((c.rows, 8, 128), 3.0, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and len(junk) == 4
    kw, vw = L.draft_layer_read(*c.cache, *c.batch, c.rows)
    assert torch.equal(kb, kw) and torch.equal(vb, vw)


def test_graph_replays(dev):
    """append and attend in a captured graph, replayed between other work."""
    c = Case(dev, [(3, 2000), (3, 90)], 8, 2, 128, 64, seed=18).upload()
    rope = torch.from_numpy(L.draft_layer_rope_table(c.max_pages * 64, 128)).to(dev)
    q, k, v = (bf16(c.rng, c.rows, h, 128).to(dev) for h in (8, 2, 2))
    ws = L.draft_layer_workspace(c.rows, 2, 8, 2, 128, dev)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((c.rows, 8), dtype=torch.float32, device=dev)

    def step():
        L.draft_layer_append(q, k, v, rope, *c.cache, *c.batch, q_out=qr)
        L.draft_layer_attend(qr, *c.cache, *c.batch, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device=dev).to(torch.bfloat16))
        before = [t.clone() for t in c.cache]
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), [t.clone() for t in c.cache]
        for t, b in zip(c.cache, before):
            t.copy_(b)
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1]), i
        assert all(torch.equal(a, b) for a, b in zip(c.cache, got[2])), i


def test_offsets_past_32_bits(dev):
    """Pages beyond the 4 GiB mark of the code arrays."""
    hkv, d, page = 8, 256, 256
    n_pages = (1 << 32) // (hkv * d * page) + 3
    codes = [torch.full((n_pages, hkv, page, d), 128, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.ones((n_pages, hkv), device=dev) for _ in range(2)]
    rng = np.random.default_rng(19)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=dev)
    start, length = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, 300], [300]))
    q, k, v = (bf16(rng, 300, hkv, d) for _ in range(3))
    L.draft_layer_append(None, k.to(dev), v.to(dev), None, *codes, *scales, start, length, table)
    kb, vb = L.draft_layer_read(*codes, *scales, start, length, table, 300)
    for got, x in ((kb, k), (vb, v)):
        assert (got.float().cpu() - x.float()).abs().max() <= x.float().abs().max() / 127 * 0.51 + 0.02
    out, _ = L.draft_layer_attend(q.to(dev), *codes, *scales, start, length, table)
    z = torch.matmul(q.float().transpose(0, 1), kb.float().cpu().permute(1, 2, 0).contiguous()) / 16
    z = z.masked_fill(torch.ones(300, 300, dtype=torch.bool).triu(1), float("-inf"))
    want = torch.matmul(z.softmax(-1), vb.float().cpu().transpose(0, 1).contiguous()).transpose(0, 1)
    # the read-back values are rounded to bf16 (2^-8 of z's and v's terms), which the cache's are not
    assert (out.float().cpu() - want).abs().max() <= 0.05


def test_binding_refuses(dev):
    c = Case(dev, [(2, 40)], 4, 2, 64, 32, seed=20).upload()
    q = c.q.to(dev)
    bad = [
        dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[:, :, :32]), dict(q=q.cpu()), dict(k=c.cache[0][:, :, :, :32]),
        dict(k=c.cache[0].to(torch.int8)), dict(ks=c.cache[2].double()), dict(ks=c.cache[2][:1]), dict(start=c.batch[0].long()),
        dict(start=c.batch[0][:1]), dict(length=c.batch[1][:0]), dict(table=c.batch[2].cpu()), dict(out=torch.empty((2, 4, 64), device=dev)),
        dict(lse=torch.empty((2, 3), device=dev)), dict(workspace=torch.zeros(64, dtype=torch.uint8, device=dev)), dict(scale=-1.0)]
    for change in bad:
        a = {**dict(q=q, k=c.cache[0], v=c.cache[1], ks=c.cache[2], vs=c.cache[3], start=c.batch[0], length=c.batch[1], table=c.batch[2]),
             **{x: y for x, y in change.items() if x not in ("out", "lse", "workspace", "scale")}}
        with pytest.raises(ValueError):
            L.draft_layer_attend(*a.values(), **{x: y for x, y in change.items() if x in ("out", "lse", "workspace", "scale")})
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=dev)
    for change in (dict(k=k[:1]), dict(v=k[:, :1]), dict(rope=torch.zeros((8, 32, 2), device=dev)), dict(rope=torch.zeros((640, 65, 2), device=dev))):
        a = {**dict(q=q, k=k, v=k, rope=None), **change}
        with pytest.raises(ValueError):
            L.draft_layer_append(*a.values(), *c.cache, *c.batch)


@pytest.mark.parametrize("window,sinks", [(0, 0), (96, 4)])
def test_example_runs(dev, window, sinks):
    """The draft step with cache and head together: the same drafts twice, all of them tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    kw = dict(seqs=3, prompt=150, slots=4, rounds=2, hidden=512, vocab=3000, hq=5, hkv=1, d=64, page=32, window=window, sinks=sinks,
              say=lambda *_: None)
    a, b = mod.run(**kw), mod.run(**kw)
    assert a.shape == (2, 3, 4) and int(a.min()) >= 0 and int(a.max()) < 3000
    assert torch.equal(a, b)


@pytest.mark.parametrize("lens,d", [([(1, 9000)], 128), ([(9, 4000)] * 3, 128), ([(700, 4000), (100, 100)], 64), ([(1, 300 * i + 1) for i in range(30)], 256)])
def test_workspace_may_hold_anything_after_its_counters(dev, lens, d):
    """Parts are read only where this call wrote them."""
    c = Case(dev, lens, 8, 2, d, 64, seed=23).upload()
    ws = torch.full((L.draft_layer_workspace_bytes(c.rows, len(lens), 8, 2, d),), 255, dtype=torch.uint8, device=dev)   # NaN as fp32
    ws[:L.WORKSPACE_ZERO_BYTES] = 0
    for _ in range(2):
        check_attend(c, 0, 0, workspace=ws)
        assert not ws[:L.WORKSPACE_ZERO_BYTES].any()
        ws[L.WORKSPACE_ZERO_BYTES:] = 255


@pytest.mark.parametrize("new,d", [(1, 64), (9, 128), (40, 64), (200, 128), (30, 256)])
@pytest.mark.parametrize("power", [10, 28, 31, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_attend_large_scores(dev, new, d, power, sign):
    """Scores of 2^power, past what fp32 holds to a unit: one token stands out by a
    quarter of them, far more than their rounding, so every row is that token's
    value; lower than all of -1e30, scores are still scores."""
    c = Case(dev, [(new, 700)], 4, 2, d, 64, seed=24)
    signs = c.rng.choice([-1.0, 1.0], d)
    far = 100 if sign > 0 else -80         # codes along the signs: the others', and the winner's 25% to 40% above
    win = 127 if sign > 0 else -40
    for t in range(700):
        code = (128 + signs * (win if t == 130 else far)).astype(np.uint8)
        c.kc[c.table[0, t // 64]].reshape(2, -1)[:, O.key_byte(np.full(d, t % 64), np.arange(d), d)] = code
    c.ks[:] = 2.0 ** (power // 2)
    c.q = torch.from_numpy(np.tile(signs * 2.0 ** (power - power // 2 - 6), (new, 4, 1)).astype(np.float32)).to(torch.bfloat16)
    c.upload()
    out, lse = check_attend(c, 0, 0, scale=1.0 / d)
    _, vn = c.naturals()
    pid = c.table[0, 2]
    want = np.repeat(vn[pid, :, 130 % 64] * c.vs[pid].astype(np.float64)[:, None], 2, axis=0)
    assert np.all(np.abs(out - want) <= half_ulp(want) + 2.0 ** -11 * np.abs(want))
    z = 2.0 ** (power - 6) * win
    assert np.all(np.abs(lse - z) <= (d + 16) * U * abs(z))


@pytest.mark.parametrize("new,d", [(3, 64), (9, 128), (40, 64), (200, 128), (30, 256)])
def test_attend_infinite_query_is_nan(dev, new, d):
    """An infinite element makes the row NaN even where every score is -inf."""
    c = Case(dev, [(new, 700)], 4, 2, d, 64, seed=25)
    c.kc[:] = np.minimum(c.kc, 127)                      # negative codes alone
    c.upload()
    out, lse = check_attend(c, 0, 0)
    q = c.q.clone()
    q[1, 2, :] = 0.0
    q[1, 2, 5] = float("inf")
    got, glse = (t.double().cpu().numpy() for t in L.draft_layer_attend(q.to(dev), *c.cache, *c.batch))
    bad = np.zeros((new, 4), bool)
    bad[1, 2] = True
    assert np.isnan(got[bad]).all() and np.isnan(glse[bad]).all()
    assert np.array_equal(got[~bad], out[~bad]) and np.array_equal(glse[~bad], lse[~bad])


@pytest.mark.parametrize("new,length,d,window,sinks", [(5, 130, 64, 0, 0), (40, 600, 128, 0, 0), (260, 600, 64, 0, 0), (40, 600, 256, 100, 4),
                                                       (1, 5000, 128, 0, 0), (9, 5000, 64, 0, 0)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_attend_scale_not_finite(dev, new, length, d, window, sinks, which, value):
    """A page whose scale is not finite makes the rows that see it NaN, and no other row."""
    page = 32
    c = Case(dev, [(new, length)], 4, 2, d, page, seed=26).upload()
    out, lse = check_attend(c, window, sinks)
    pos = np.arange(length - new, length)
    for j in {(length - 1) // page, (length - new) // page, 2, 0}:
        c.upload()
        c.cache[2 if which == "k" else 3][int(c.table[0, j]), 1] = value
        got, glse = (t.double().cpu().numpy() for t in L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch, window=window, sinks=sinks))
        t = np.arange(j * page, min(j * page + page, length))[None, :]
        seen = t <= pos[:, None]
        if window:
            seen &= (t > pos[:, None] - window) | (t < sinks)
        bad = np.zeros((new, 4), bool)
        bad[:, 2:] = seen.any(axis=1)[:, None]
        assert np.isnan(got[bad]).all() and np.isnan(glse[bad]).all(), j
        assert np.array_equal(got[~bad], out[~bad]) and np.array_equal(glse[~bad], lse[~bad]), j


@pytest.mark.parametrize("new,length,d,page", [(3, 40, 64, 32), (9, 100, 128, 64), (200, 230, 64, 64), (300, 300, 256, 256)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_append_not_finite(dev, new, length, d, page, value):
    """A new value that is no number makes its page and head NaN, reading and
    attention say so, tokens that follow there do not undo it, a fresh start does."""
    rope = torch.from_numpy(L.draft_layer_rope_table(-(-length // page) * page + 2 * page, d)).to(dev)
    for which in ("k", "v"):
        c = Case(dev, [(new, length)], 4, 2, d, page, seed=27).upload()
        kv = {x: bf16(c.rng, new, 2, d).to(dev) for x in "kv"}
        begin, at = length - new, new - 2
        pid = int(c.table[0, (begin + at) // page])
        L.draft_layer_append(None, kv["k"], kv["v"], rope, *c.cache, *c.batch)
        clean = [t.clone() for t in c.cache]
        clean_kv = L.draft_layer_read(*c.cache, *c.batch, new)
        before = L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch)
        c.upload()
        kv[which][at, 1, d // 2 + 3] = value
        L.draft_layer_append(None, kv["k"], kv["v"], rope, *c.cache, *c.batch)
        scale, other = (c.cache[2], c.cache[3]) if which == "k" else (c.cache[3], c.cache[2])
        want = (clean[2] if which == "k" else clean[3]).clone()
        want[pid, 1] = float("nan")
        assert torch.equal(scale.isnan(), want.isnan()) and torch.equal(scale.nan_to_num(), want.nan_to_num())
        assert torch.equal(other, clean[3] if which == "k" else clean[2])
        got_kv = L.draft_layer_read(*c.cache, *c.batch, new)
        on_page = torch.arange(begin, length, device=dev) // page == (begin + at) // page
        for x, got, was in (("k", got_kv[0], clean_kv[0]), ("v", got_kv[1], clean_kv[1])):
            nan = torch.zeros_like(got, dtype=torch.bool)
            if x == which:
                nan[on_page, 1] = True
            assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], was[~nan])
        out, lse = L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch)
        see = torch.arange(begin, length, device=dev) >= (begin + at) // page * page
        nan = torch.zeros_like(lse, dtype=torch.bool)
        nan[:, 2:] = see[:, None]
        assert torch.equal(lse.isnan(), nan) and bool(out[nan].isnan().all())
        assert torch.equal(out[~nan], before[0][~nan]) and torch.equal(lse[~nan], before[1][~nan])
        # one more token of the page: still NaN; the page's own start: no longer
        one = torch.tensor([0, 1], dtype=torch.int32, device=dev)
        fine = {x: bf16(c.rng, 1, 2, d).to(dev) for x in "kv"}
        first = (begin + at) // page * page
        for position, still in ((first + 1, True), (first, False)):
            L.draft_layer_append(None, fine["k"], fine["v"], rope, *c.cache, one, torch.tensor([position + 1], dtype=torch.int32, device=dev), c.batch[2])
            assert bool(scale[pid, 1].isnan()) == still and not bool(scale[pid, 0].isnan())


def test_append_not_finite_in_queries_alone(dev):
    """The queries' own NaN and infinity stay in their rows and heads and out of the cache."""
    c = Case(dev, [(9, 100)], 4, 2, 64, 32, seed=28).upload()
    rope = torch.from_numpy(L.draft_layer_rope_table(160, 64)).to(dev)
    k, v = bf16(c.rng, 9, 2, 64).to(dev), bf16(c.rng, 9, 2, 64).to(dev)
    q = c.q.to(dev)
    clean = L.draft_layer_append(q, k, v, rope, *c.cache, *c.batch)
    kept = [t.clone() for t in c.cache]
    q[4, 3, 7], q[6, 0, 1] = float("nan"), float("inf")
    got = L.draft_layer_append(q, k, v, rope, *c.upload().cache, *c.batch)
    nan = torch.zeros((9, 4), dtype=torch.bool, device=dev)
    nan[4, 3] = nan[6, 0] = True
    assert torch.equal(got[~nan], clean[~nan]) and not bool(torch.isfinite(got[nan]).all(dim=1).any())
    assert all(torch.equal(a, b) for a, b in zip(kept, c.cache))


@pytest.mark.parametrize("new", [3, 60])
def test_append_limits_are_attends(dev, new):
    """The largest values that append takes, rotated by the largest entries, next
    to pages of the smallest scale: attend holds over what append leaves."""
    d, page, length = 128, 32, 200
    c = Case(dev, [(length, length)], 4, 2, d, page, seed=29)
    c.upload()
    rope = L.draft_layer_rope_table(c.max_pages * page, d, mscale=3.99)
    assert np.abs(rope).max() < 4
    big = 2.0 ** 60 * (1 - 2.0 ** -8)
    k, v = (torch.from_numpy(c.rng.choice([-big, big], (length, 2, d)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    k[32:64], v[64:96] = 0.0, 0.0
    before = c.naturals()
    q = torch.from_numpy(c.rng.choice([-big, big], (length, 4, d)).astype(np.float32)).to(torch.bfloat16)
    c.q = q
    got = L.draft_layer_append(q.to(dev), k.to(dev), v.to(dev), torch.from_numpy(rope).to(dev), *c.cache, *c.batch)
    check_append(c, None, rope, False, k, v, before, with_q=False)
    want, _ = O.append(q.float().numpy(), k.float().numpy(), v.float().numpy(), rope, *before, c.ks, c.vs, c.q_start, c.kv_len, c.table, False)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= half_ulp(want) + 4 * 8 * U * big)      # entries of 4 instead of 1
    assert 2.0 ** 62 < float(got.float().abs().max()) < 2.0 ** 63
    c.kc, c.vc, c.ks, c.vs = (t.cpu().numpy() for t in c.cache)
    used = c.table[0, :-(-length // page)]
    assert c.ks[used].max() > 2.0 ** 55 and max(c.ks[used].max(), c.vs[used].max()) < 2.0 ** 57
    assert c.ks[used].min() == c.vs[used].min() == 2.0 ** -40
    # rows whose scores stay in single figures, then the rotated queries themselves
    c.q_start[1] = c.rows = new
    c.q = (got.float() * 2.0 ** -126)[length - new:].to(torch.bfloat16).cpu()
    c.upload()
    check_attend(c, 0, 0)
    c.q = got[length - new:].cpu()
    check_attend(c, 0, 0, scale=2.0 ** -14)


def test_append_rejected_outlier(dev):
    """A rejected token far larger than its page's: written over, it is gone, but the
    step that it raised stays with the page's accepted tokens and with those that
    follow there; pages before it, and its own once it starts afresh, are as if it
    had never been."""
    d, page = 64, 32
    c = Case(dev, [(1, 1)], 1, 1, d, page, seed=30, max_pages=3, spare=4)
    c.table[0] = [0, 1, 2]
    c.upload()
    one = lambda n: torch.tensor([n], dtype=torch.int32, device=dev)  # noqa: E731
    start = lambda n: torch.tensor([0, n], dtype=torch.int32, device=dev)  # noqa: E731
    put = lambda x, end: L.draft_layer_append(None, x.to(dev), x.to(dev), None, *c.cache, start(len(x)), one(end), c.batch[2])  # noqa: E731
    x = bf16(c.rng, 48, 1, d)
    put(x[:42], 42)                                          # positions 0..41: ten accepted tokens on page 1
    own = c.cache[3][:2, 0].clone()
    first = L.draft_layer_read(*c.cache, start(42), one(42), c.batch[2], 42)[1]
    put(x[42:43] * 100.0, 43)                                # an outlier, rejected
    raised = float(c.cache[3][1, 0])
    assert raised > 20 * float(own[1]) and c.cache[3][0, 0] == own[0]
    put(x[42:48], 48)                                        # what took its place
    assert float(c.cache[3][1, 0]) == raised
    got = L.draft_layer_read(*c.cache, start(48), one(48), c.batch[2], 48)[1]
    assert torch.equal(got[:32], first[:32])                 # the page before
    err = (got.float().cpu() - x.float()).abs().flatten(1).max(dim=1).values
    read = float(half_ulp(8.0))                              # what is read back is below 8
    lim = torch.full((48,), (0.5 + 2.0 ** -12) * raised + read)
    lim[32:42] += 0.5 * float(own[1])                        # rounded twice
    assert bool((err[32:] <= lim[32:]).all())
    put(x[32:48], 48)                                        # from its token 0 on
    again = L.draft_layer_read(*c.cache, start(48), one(48), c.batch[2], 48)[1]
    assert float(c.cache[3][1, 0]) == np.float32(x[32:48].float().abs().max().item()) / np.float32(127)
    assert float((again.float().cpu() - x.float()).abs().max()) <= (0.5 + 2.0 ** -12) * float(c.cache[3][:2].max()) + read


@pytest.mark.parametrize("hkv,new,seqs,window", [(8, 1, 30, 0), (2, 1, 30, 0), (2, 3, 100, 0), (8, 2, 70, 500), (1, 1, 3, 0), (7, 1, 40, 0)])
def test_attend_large_heads_of_few_rows(dev, hkv, new, seqs, window):
    """The streaming kernel at heads of 256 over several sequences, whose fewer
    workgroups take other runs and parts: lengths far apart, in each plan."""
    lens = [(new if i % 7 else 0, new + 3 + (95 * i) % 2500) for i in range(seqs)]
    lens[1] = (new, 5000)
    check_attend(Case(dev, lens, hkv * 2, hkv, 256, 64, seed=31 + hkv).upload(), window, 4 if window else 0)


@pytest.mark.parametrize("lens", [[(9, 100), (1, 40)], [(80, 200)]])
def test_rows_of_no_sequence_are_left_alone(dev, lens):
    """A batch with more rows than its sequences have: the others' outputs stay as
    they are, and the covered ones' are those of the batch without them."""
    c = Case(dev, lens, 4, 2, 64, 32, seed=32).upload()
    n, extra = c.rows, 50
    want = L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch)
    q = torch.cat([c.q, torch.full((extra, 4, 64), float("nan"), dtype=torch.bfloat16)]).to(dev)
    out = torch.full((n + extra, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((n + extra, 4), 7.0, device=dev)
    L.draft_layer_attend(q, *c.cache, *c.batch, out=out, lse=lse)
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())
    assert torch.allclose(out[:n].float(), want[0].float(), rtol=2.0 ** -7, atol=2.0 ** -8)     # perhaps in tiles of another height
    assert torch.allclose(lse[:n], want[1], rtol=0, atol=2.0 ** -12)
    read = L.draft_layer_read(*c.cache, *c.batch, n)
    k, v = (torch.full((n + extra, 2, 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    L.draft_layer_read(*c.cache, *c.batch, n + extra, k_out=k, v_out=v)
    assert all(torch.equal(a[:n], b) and bool((a[n:] == 7).all()) for a, b in ((k, read[0]), (v, read[1])))
    # append: the rows without a sequence write nothing to the cache
    kk, vv = (torch.cat([bf16(c.rng, n, 2, 64), torch.full((extra, 2, 64), float("nan"), dtype=torch.bfloat16)]).to(dev) for _ in range(2))
    rope = torch.from_numpy(L.draft_layer_rope_table(c.max_pages * 32, 64)).to(dev)
    first = L.draft_layer_append(q[:n], kk[:n], vv[:n], rope, *c.cache, *c.batch)
    kept = [t.clone() for t in c.cache]
    both = L.draft_layer_append(q, kk, vv, rope, *c.upload().cache, *c.batch)
    assert torch.equal(both[:n], first) and all(torch.equal(a, b) for a, b in zip(kept, c.cache))
