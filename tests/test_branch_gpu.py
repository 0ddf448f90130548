"""The operators on several branches on the GPU against the oracle.

Attention: the tolerances of draft_layer_attend's tests (z's products and sums, weights of
11 bits, bf16's half ulp; their 2^-18 and 2^-20 hold the joining of the parts too).

Pages are moved, not computed: tables, counts and every byte of the pool are
compared as they are.

Log probabilities, from the arithmetic (u = 2^-24, one fp32 rounding; d = z - max z
of an element, E the mean under the row's probabilities):
  exponent       f log2(e) is two roundings (its constant's and the product's), x - max
                 one, their product one: 4 u |d|
  weight         that, and 2^-22 for the exponential
  sums           of positive terms, each through at most N/2048 + 8 additions a lane, 8 over
                 the lanes, 3 over the waves and one a part (each joining rounds its weight
                 too): A = (N/2048 + 3 * (20 + parts)) u relative, beside the weights' own
  lse            4 u E|d| + 2^-22 + A, u |f max| for f max, and u |lse|, 2 u ln(sum) for the logarithm
  logprob        3 u |d_token| and lse's without f max
  entropy        ln(sum)'s as lse's; s/l: (2^-22 + A) E|d| twice (s and l), 4 u E d^2 and 8 u E|d|
"""
import numpy as np
import pytest

from bit_quantized_lm_amd import _binding as B
from bit_quantized_lm_amd import _branch as R
from bit_quantized_lm_amd import _layer as L
from oracle import branch as O
from oracle import layer as OL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    B.load_library()
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)


# --------------------------------------------------------------------- pages
class Pool:
    """A pool of random contents, some of it in use by the sequences of a table."""

    def __init__(self, dev, lens, n_pages, hkv, d, page, seed, reserve=0, shared=0, wide=None):
        """shared: every second sequence has that many full pages from the one before it."""
        rng = self.rng = np.random.default_rng(seed)
        self.dev, self.page, self.n_pages = dev, page, n_pages
        self.kv_len = np.array(lens, np.int32)
        held = [-(-(n + reserve) // page) for n in lens]
        self.wide = wide or max(max(held), 1) + 1
        self.table = np.full((len(lens), self.wide), -1, np.int32)
        order, at = rng.permutation(n_pages), 0
        for s, n in enumerate(held):
            k = min(shared, lens[s] // page, lens[s - 1] // page) if s % 2 else 0
            self.table[s, :k] = self.table[s - 1, :k]
            self.table[s, k:n] = order[at:at + n - k]
            at += n - k
        self.uses = np.bincount(self.table[self.table >= 0], minlength=n_pages).astype(np.int32)
        g = torch.Generator(device=dev).manual_seed(seed)
        shape = (n_pages, hkv, page, d)
        self.cache = [torch.randint(0, 256, shape, dtype=torch.uint8, generator=g, device=dev) for _ in range(2)]
        self.cache += [torch.rand(shape[:2], generator=g, device=dev) for _ in range(2)]

    def fork(self, parents, need, **kw):
        before = [t.clone() for t in self.cache]
        got = R.draft_branch_fork(*self.cache, ints(self.uses, self.dev), ints(self.table, self.dev), ints(self.kv_len, self.dev),
                                  ints(parents, self.dev), ints(need, self.dev), **kw)
        torch.cuda.synchronize()
        table, uses, status, copies = O.fork(self.uses, self.table, self.kv_len, parents, need, self.page)
        assert np.array_equal(got[2].cpu().numpy(), status)
        assert np.array_equal(got[1].cpu().numpy(), uses) and np.array_equal(got[0].cpu().numpy(), table)
        self.moved(before, copies)
        return table, uses, status, copies

    def compact(self, **kw):
        before = [t.clone() for t in self.cache]
        got = R.draft_branch_compact(*self.cache, ints(self.uses, self.dev), ints(self.table, self.dev), **kw)
        torch.cuda.synchronize()
        table, uses, status, moves = O.compact(self.uses, self.table)
        assert np.array_equal(got[2].cpu().numpy(), status)
        assert np.array_equal(got[1].cpu().numpy(), uses) and np.array_equal(got[0].cpu().numpy(), table)
        self.moved(before, moves)
        return table, uses, status, moves

    def moved(self, before, moves):
        for was, now in zip(before, self.cache):
            for a, b in moves:
                was[b].copy_(was[a])
            assert torch.equal(was, now)


FORKS = [
    # lens, new rows' parents, tokens more, pages, hkv, d, page, reserve, shared
    ([1], [0], 1, 3, 1, 64, 32, 0, 0),
    ([33], [0, 0, 0], 9, 20, 8, 128, 64, 9, 0),
    ([100, 64, 7], [0, 0, 1, 1, 2], 1, 30, 2, 128, 64, 1, 0),            # one ends on a page's last token
    ([100, 64, 7], [2, -1, 0, 2, 99, 0], 40, 60, 3, 64, 32, 0, 0),       # none, in no order, outside
    ([500, 500, 300], [1, 1], 5, 80, 2, 256, 32, 16, 7),                 # two end; pages shared with one that does not go on
    ([0, 5], [0, 1, 0], 0, 6, 1, 64, 32, 0, 0),                          # an empty sequence; nothing needed
    ([256 * 3 + 1] * 5, [4, 3, 2, 1, 0, 0, 1], 300, 60, 1, 256, 256, 255, 2),
    ([31 * (i % 9) + 1 for i in range(90)], [i // 3 for i in range(200)], 12, 2500, 1, 64, 32, 6, 1),
    ([70, 200, 40], [0, 0, 1, -1, 1], 900, 300, 1, 64, 32, 500, 2),      # many pages kept, many taken
    ([20 * (i % 9) + 1 for i in range(90)], [i // 3 for i in range(250)], 7, 2048, 1, 64, 32, 6, 1),
]


@pytest.mark.parametrize("spare", [0, 2500])      # one chunk of counts and several
@pytest.mark.parametrize("lens,parents,more,n_pages,hkv,d,page,reserve,shared", FORKS)
def test_fork(dev, lens, parents, more, n_pages, hkv, d, page, reserve, shared, spare):
    n_pages += spare
    p = Pool(dev, lens, n_pages, hkv, d, page, seed=len(parents) + d, reserve=reserve, shared=shared, wide=max(lens) // page + more // page + 4)
    need = [lens[q] + more if 0 <= q < len(lens) else more + 3 for q in parents]
    _, _, status, _ = p.fork(parents, need)
    assert status[1] == 0
    p.fork(parents, need, workspace=torch.full((R.draft_branch_pages_workspace_bytes(n_pages, len(parents)),), 255, dtype=torch.uint8, device=dev))


def test_fork_long_rows(dev):
    """Rows of more entries than a workgroup has threads, all fresh, kept or shared, over several chunks of counts."""
    p = Pool(dev, [32 * 700 + 5, 40], 6100, 1, 64, 32, seed=3, reserve=32 * 400, wide=1500)
    _, _, status, copies = p.fork([0, 0, -1, 1], [32 * 1400, 32 * 1100, 32 * 1500, 32 * 600])
    assert status[1] == 0 and len(copies) == 1


def test_fork_many_rows(dev):
    """As many rows as a table may have."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(0, 90, 4096)]
    p = Pool(dev, lens, 30000, 1, 64, 32, seed=4, reserve=3, wide=5)
    parents = rng.integers(-1, 4096, 4096)
    _, _, status, copies = p.fork(parents, [lens[q] + 4 if q >= 0 else 20 for q in parents])
    assert status[1] == 0 and len(copies) > 500


@pytest.mark.parametrize("spare", [0, 2500])
def test_fork_lacking_pages_does_nothing(dev, spare):
    p = Pool(dev, [100, 40], 9 + spare, 2, 64, 32, seed=5, reserve=1)
    p.uses[np.nonzero(p.uses == 0)[0][3:]] = 2
    table, uses, status, copies = p.fork([0, 0, 1, 1], [130, 130, 60, 60])
    assert status[1] == 1 and status[0] == 3 and not copies and (table == -1).all() and np.array_equal(uses, p.uses)
    p.fork([0, 1, 1], [104, 60, 60])       # what is left suffices for this


@pytest.mark.parametrize("spare", [0, 2500])
def test_fork_odd_numbers(dev, spare):
    """Lengths, needs, ids and counts that no caller should have: taken as the header says."""
    p = Pool(dev, [100, 64, 90, 20], 60 + spare, 1, 64, 32, seed=6, wide=5)
    p.kv_len[:] = [-5, 1 << 30, 90, 20]
    p.table[1, 2:] = [-7, 60 + spare, 1 << 30]     # no page
    p.table[2, 2] = -1                     # the partial page is missing
    p.uses[p.table[3, 0]] = 3              # something else keeps it
    p.uses[p.uses == 0] = np.where(np.arange((p.uses == 0).sum()) % 3 == 0, -2, 0)
    p.fork([0, 1, 2, 2, 3, 3, 4, -(1 << 31), (1 << 31) - 1], [-9, 1 << 30, 95, 0, 21, 200, 33, -1, (1 << 31) - 1])


@pytest.mark.parametrize("spare", [0, 2500])
def test_fork_keeps_no_page_that_is_shared(dev, spare):
    """A page that a sequence has from another is copied before it is written, for its first row too."""
    p = Pool(dev, [64, 64], 12 + spare, 1, 64, 32, seed=7, shared=2)
    p.kv_len[:] = [40, 64]                 # the first went back behind what the second has from it
    _, _, _, copies = p.fork([0, 1], [60, 70])
    assert [a for a, _ in copies] == [p.table[0, 1]]


@pytest.mark.parametrize("n_pages,hkv,d,page,lens", [
    (1, 1, 64, 32, [1]), (7, 1, 64, 32, [5, 60]), (60, 3, 128, 64, [500, 64, 1, 700]), (60, 2, 256, 256, [1000, 2000, 30]),
    (2048, 1, 64, 32, [100 * i for i in range(20)]), (5000, 1, 64, 32, [2000 + 300 * (i % 7) for i in range(40)])])
def test_compact(dev, n_pages, hkv, d, page, lens):
    p = Pool(dev, lens, n_pages, hkv, d, page, seed=n_pages, shared=1)
    table, uses, status, moves = p.compact()
    assert (uses[:status[0]] > 0).all() and not uses[status[0]:].any()
    # drawn together already: nothing moves
    p.uses, p.table = uses, table
    assert not p.compact()[3]


@pytest.mark.parametrize("n", [30, 2048, 5000])
def test_compact_all_or_none_in_use(dev, n):
    p = Pool(dev, [100], n, 1, 64, 32, seed=8, wide=30)
    p.uses[:] = 1
    assert not p.compact()[3]
    p.uses[:] = 0
    assert not p.compact()[3]
    p.uses[:n // 2], p.uses[n // 2:] = -1, 2
    assert len(p.compact()[3]) == n // 2
    p.table[0, :3] = [-9, n, 1 << 30]     # no page: left as they are
    p.compact()


def test_pages_of_a_large_pool(dev):
    """More chunks of counts than a workgroup has threads."""
    n = 2048 * 260 + 3
    p = Pool(dev, [40], 8, 1, 64, 32, seed=9, wide=8)
    cache = [torch.zeros((n, 1, 32, 64), dtype=torch.uint8, device=dev) for _ in range(2)]
    cache += [torch.zeros((n, 1), dtype=torch.float32, device=dev) for _ in range(2)]
    uses = (p.rng.random(n) < 0.6).astype(np.int32)
    uses[:2048 * 258] = 1                  # the free ones stand at the end
    used = np.nonzero(uses)[0]
    table = used[p.rng.integers(0, len(used), (3, 50))].astype(np.int32)
    kv_len = np.array([40 * 32 + 3, 20, 0], np.int32)
    args = (ints(uses, dev), ints(table, dev))
    cache[0][torch.from_numpy(table[0, 40:41]).long().to(dev)] = 7
    got = R.draft_branch_fork(*cache, *args, ints(kv_len, dev), ints([0, 0, -1], dev), ints([1400, 1500, 64], dev))
    want = O.fork(uses, table, kv_len, [0, 0, -1], [1400, 1500, 64], 32)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    assert want[3] and all(bool((cache[0][b] == 7).all()) for _, b in want[3])
    got = R.draft_branch_compact(*cache, *args)
    want = O.compact(uses, table)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want)) and len(want[3]) > 500


@pytest.mark.parametrize("n_pages", [60, 2500])
def test_pages_with_counts_at_any_alignment(dev, n_pages):
    p = Pool(dev, [100, 64, 300], n_pages, 1, 64, 32, seed=13, reserve=3)
    parents, need = [0, 0, 2, 1, 2], [110, 120, 310, 70, 340]
    want, packed = O.fork(p.uses, p.table, p.kv_len, parents, need, 32), O.compact(p.uses, p.table)
    for off in range(1, 4):
        uses = torch.zeros(n_pages + off, dtype=torch.int32, device=dev)[off:]
        uses.copy_(ints(p.uses, dev))
        cache = [t.clone() for t in p.cache]
        got = R.draft_branch_fork(*cache, uses, ints(p.table, dev), ints(p.kv_len, dev), ints(parents, dev), ints(need, dev))
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
        got = R.draft_branch_compact(*cache, uses, ints(p.table, dev))
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, packed))


def test_pages_refuse_overlaps(dev):
    p = Pool(dev, [40, 70], 20, 1, 64, 32, seed=10)
    uses, table = ints(p.uses, dev), ints(p.table, dev)
    two = ints([0, 1], dev)
    with pytest.raises(ValueError):
        R.draft_branch_fork(*p.cache, uses, table, ints(p.kv_len, dev), two, two, uses_out=uses)
    with pytest.raises(ValueError):
        R.draft_branch_fork(*p.cache, uses, table, ints(p.kv_len, dev), two, two, table_out=table)
    with pytest.raises(ValueError):
        R.draft_branch_compact(*p.cache, uses, table, table_out=table)
    with pytest.raises(ValueError):
        R.draft_branch_fork(*p.cache, uses, table, ints(p.kv_len, dev), two, ints([1], dev))
    with pytest.raises(ValueError):
        R.draft_branch_fork(*p.cache, uses, table.long(), ints(p.kv_len, dev), two, two)


@pytest.mark.parametrize("n_pages", [90, 4200])
def test_pages_on_another_stream_and_in_a_graph(dev, n_pages):
    p = Pool(dev, [100, 500, 64, 7], n_pages, 2, 128, 32, seed=11, reserve=5)
    parents, need = [0, 1, 1, 2, 3, 3], [110, 530, 520, 70, 40, 40]
    args = [ints(x, dev) for x in (p.uses, p.table, p.kv_len, parents, need)]
    want = O.fork(p.uses, p.table, p.kv_len, parents, need, 32)
    packed = O.compact(p.uses, p.table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = R.draft_branch_fork(*p.cache, *args, stream=side)
    side.synchronize()
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    ws = R.draft_branch_pages_workspace(n_pages, 6, dev)
    outs = [torch.empty_like(t) for t in got]
    more = [torch.empty_like(args[1]), torch.empty_like(args[0]), torch.empty_like(outs[2])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.draft_branch_fork(*p.cache, *args, table_out=outs[0], uses_out=outs[1], status=outs[2], workspace=ws)
        R.draft_branch_compact(*p.cache, args[0], args[1], table_out=more[0], uses_out=more[1], status=more[2], workspace=ws)
    for i in range(3):
        for t in outs + more:
            t.fill_(77)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs, want))
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(more, packed))


# ----------------------------------------------------------------- attention
def half_ulp(x):
    """Half a bf16 ulp at x, with room for a neighbour one binade up."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -120) * (1 + 2.0 ** -8))) - 8)


class Branches:
    """A cache with random contents and a batch whose groups share prefixes.
    groups: [(prefix, [(new, tokens from the prefix's end on)])]; loose: [(new, tokens)]."""

    def __init__(self, dev, groups, loose, hq, hkv, d, page, seed, max_pages=None, members_know=True, wide=False, quick=False):
        """wide: a table with room for more tokens than what is short; quick: codes that are all alike likely."""
        rng = self.rng = np.random.default_rng(seed)
        self.dev, self.hq, self.hkv, self.d, self.page = dev, hq, hkv, d, page
        lens = [(n, p + t, p, i == 0) for p, m in groups for i, (n, t) in enumerate(m)] + [(n, t, 0, True) for n, t in loose]
        reach = max([t for _, t, _, _ in lens] + [p for p, _ in groups] + [1])
        self.max_pages = max_pages or max(-(-reach // page) + 1, (4096 // page + 3) * wide)
        n_pages = sum(-(-max(t, p) // page) for _, t, p, _ in lens) + 3
        order, at = rng.permutation(n_pages), 0
        self.table = np.full((len(lens), self.max_pages), -7, np.int32)
        for s, (_, total, prefix, first) in enumerate(lens):
            if first:
                leader, k = s, 0
            else:      # whole pages of the prefix are the first's, its last part is not
                k = min(prefix // page, self.max_pages)
                if members_know:
                    self.table[s, :k] = self.table[leader, :k]
            n = min(-(-max(total, prefix if first else 0) // page), self.max_pages)
            if n > k:
                self.table[s, k:n] = order[at:at + n - k]
                at += n - k
        self.q_start = np.concatenate([[0], np.cumsum([n for n, _, _, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([t for _, t, _, _ in lens], np.int32)
        self.group_start = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])]).astype(np.int32)
        self.prefix_len = np.array([p for p, _ in groups], np.int32)
        self.rows = int(self.q_start[-1])
        shape = (n_pages, hkv, page, d)
        self.codes = [rng.integers(1, 256, shape, dtype=np.uint8) if quick else
                      (np.clip(np.rint(rng.standard_normal(shape) * 33), -127, 127) + 128).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.uniform(0.01, 0.06, shape[:2]).astype(np.float32) for _ in range(2)]
        self.q = torch.from_numpy(rng.standard_normal((self.rows, hq, d)).astype(np.float32)).to(torch.bfloat16)

    def upload(self):
        self.cache = [torch.from_numpy(a).to(self.dev) for a in (*self.codes, *self.scales)]
        self.batch = [ints(a, self.dev) for a in (self.q_start, self.kv_len, self.table, self.group_start, self.prefix_len)]
        return self

    def check(self, window=0, sinks=0, q=None, scale=None, **kw):
        self.upload()
        qd = self.q.to(self.dev) if q is None else q
        scale = 1.0 / np.sqrt(self.d) if scale is None else scale
        out, lse = R.draft_branch_attend(qd, *self.cache, *self.batch, scale=scale, window=window, sinks=sinks, **kw)
        torch.cuda.synchronize()
        rows = self.rows
        want, lwant, spread, absqk = O.attend(self.q.float().numpy(), OL.natural(self.codes[0], OL.key_byte), OL.natural(self.codes[1], OL.value_byte),
                                              *self.scales, self.q_start, self.kv_len, self.table, self.group_start, self.prefix_len, scale, window, sinks)
        got, lgot = out[:rows].double().cpu().numpy(), lse[:rows].double().cpu().numpy()
        dz = (self.d + 16) * U * absqk
        none = np.isneginf(lwant)
        assert np.array_equal(np.isneginf(lgot), none) and not np.isnan(lgot).any()
        assert np.all(np.abs(lgot - lwant)[~none] <= (dz + 2.0 ** -20 + 4 * U * np.abs(lwant))[~none])
        err, lim = np.abs(got - want), half_ulp(want) + (2.0 ** -11 + 2 * dz[..., None] + 2.0 ** -18) * spread
        assert np.all(err <= lim), (err - lim).max()
        assert not got[none].any()
        return out, lse


ATTENDS = [
    # groups, loose, hq, hkv, d, page, window, sinks
    ([(1, [(1, 1)])], [], 1, 1, 64, 32, 0, 0),
    ([(64, [(1, 1), (1, 5), (1, 70)])], [], 5, 1, 128, 64, 0, 0),
    ([(960, [(1, 30)] * 4)], [], 40, 8, 128, 64, 0, 0),
    ([(5000, [(1, 20 + 3 * i) for i in range(9)])], [], 16, 2, 256, 128, 0, 0),
    ([(333, [(1, 40), (0, 9), (2, 2), (1, 300)]), (77, [(1, 1)]), (100, [(1, 600), (1, 2)])], [(1, 90), (2, 2)], 10, 2, 128, 64, 0, 0),
    ([(700, [(9, 20), (3, 3), (9, 100)])], [(4, 50)], 21, 3, 64, 32, 0, 0),              # the prefix ends inside a page
    ([(200, [(40, 40), (77, 300), (100, 101)])], [], 12, 3, 128, 32, 0, 0),
    ([(300, [(150, 150), (200, 450)]), (64, [(130, 130)])], [], 8, 2, 64, 64, 0, 0),
    ([(250, [(100, 120), (90, 90)])], [(30, 60)], 8, 1, 256, 64, 0, 0),
    ([(500, [(2, 30)] * 3)], [(5, 600)], 8, 1, 256, 128, 0, 0),                          # tiles of 64 and of 16 rows, heads of 256
    ([(400, [(70, 70)] * 2)], [(1, 30)] * 9, 2, 1, 128, 64, 0, 0),                        # groups of many rows, sequences of few
    ([(0, [(1, 40), (1, 7)])], [], 4, 2, 64, 32, 0, 0),                                  # no prefix
    ([(100, [(6, -40), (1, 3), (3, -100), (5, 2), (2, -96)])], [], 4, 2, 64, 32, 0, 0),  # rows within the prefix, rows that see nothing
    ([(500, [(1, 300), (1, 20)])], [(1, 50)], 4, 2, 64, 32, 100, 4),                     # a window that leaves the prefix out, or in part
    ([(1000, [(9, 60), (4, 9), (1, 700)])], [], 5, 1, 128, 64, 200, 70),
    ([(40, [(3, 200), (2, 30)])], [(2, 300)], 4, 2, 64, 32, 50, 100),                    # sinks past the prefix
    ([(300, [(90, 100), (60, 61)])], [], 6, 2, 128, 64, 1, 0),                           # a row sees itself alone
    ([(300, [(90, 100), (60, 61)])], [], 6, 2, 128, 64, 33, 3),
    ([(700, [(40, 90), (64, 64)])], [(10, 90)], 8, 1, 256, 64, 100000, 4),               # a window past everything
    ([(65, [(1, 1 + i) for i in range(90)])], [(1, 20)] * 5, 4, 1, 64, 32, 0, 0),         # more sequences than a wave has lanes
    ([(40 + i, [(1, 3), (1, 1 + i)]) for i in range(70)], [(1, 9)], 2, 1, 64, 32, 0, 0),  # and more groups
    ([(40 + i, [(1, -30 + i), (2, 1 + i)]) for i in range(70)], [(1, 9)], 2, 2, 64, 32, 45, 2),
    ([(20000, [(1, 3)] * 3)], [], 8, 1, 64, 128, 0, 0),                                   # few rows over a long prefix: many parts
    ([(3900, [(1, 30)] * 3)], [(2, 4000)], 8, 2, 64, 64, 0, 0),                           # the longest of the short
    ([(1200, [(3, 60)] * 25)], [(2, 900)], 16, 2, 256, 128, 0, 0),
    ([(3000, [(3, 60)] * 25)], [(2, 900)], 16, 2, 256, 128, 1900, 30),
]
SIX = [(9, 60), (1, 9), (0, 7), (1, 300), (3, 3), (2, 40)]
WINDOWS = [   # too many tiles to be short
    ([(130 * i + 5, SIX) for i in range(10)], [], 40, 40, 64, 32, 100, 4),
    ([(130 * i + 5, SIX) for i in range(10)], [(1, 500)] * 4, 40, 40, 64, 32, 1, 0),
    ([(300, SIX * 4), (64, SIX * 5)], [(2, 100)] * 3, 40, 20, 128, 64, 33, 3),
    ([(1000, SIX * 10)], [], 40, 20, 128, 64, 200, 70),
    ([(40, SIX * 10)], [], 20, 20, 128, 32, 50, 100),
    ([(200, [(70, 90)] * 8), (100, SIX)], [(90, 200)] * 2, 32, 8, 128, 32, 77, 0),
    ([(500, SIX * 5), (700, SIX * 4)], [(1, 900)], 20, 10, 256, 64, 150, 4),
    ([(130 * i + 5, SIX) for i in range(15)], [(1, 5)], 24, 24, 64, 32, 45, 2),
    ([(130 * i + 5, SIX) for i in range(15)], [(1, 5)], 24, 12, 128, 32, 45, 2),
    ([(130 * i + 5, SIX) for i in range(12)], [(1, 5)], 10, 10, 256, 32, 200, 2),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("groups,loose,hq,hkv,d,page,window,sinks", ATTENDS)
def test_attend(dev, groups, loose, hq, hkv, d, page, window, sinks, wide):
    Branches(dev, groups, loose, hq, hkv, d, page, seed=d + page + hq + len(groups), members_know=len(groups) % 2 == 0, wide=wide).check(window, sinks)


@pytest.mark.parametrize("groups,loose,hq,hkv,d,page,window,sinks", WINDOWS)
def test_attend_windows_of_many_tiles(dev, groups, loose, hq, hkv, d, page, window, sinks):
    c = Branches(dev, groups, loose, hq, hkv, d, page, seed=d + page + hq, wide=True)
    tiles = (c.rows * (hq // hkv) // 16 + len(c.kv_len)) * hkv
    assert tiles > {64: 2048, 128: 1024, 256: 512}[d]
    c.check(window, sinks)


@pytest.mark.parametrize("groups,loose,hq,hkv,d,page,window,sinks", [
    ([(1000, SIX * 10)], [], 48, 24, 128, 64, 200, 70),                    # up to 64 sequences
    ([(500, SIX * 5), (700, SIX * 4)], [], 32, 16, 256, 64, 150, 4),
    ([(300, SIX * 8), (64, SIX * 8)], [(2, 100)] * 3, 40, 20, 128, 64, 33, 3),      # more
    ([(40, SIX * 14)], [], 20, 20, 128, 32, 50, 100),
    ([(130 * i + 5, SIX) for i in range(18)], [(1, 5)], 10, 10, 256, 32, 200, 2),
])
def test_attend_windows_planned(dev, groups, loose, hq, hkv, d, page, window, sinks):
    """Tiles of sequences of equal rows, by which a batch with a window is too large for one launch."""
    c = Branches(dev, groups, loose, hq, hkv, d, page, seed=d + page + hq, wide=True)
    rows = -(-c.rows * (hq // hkv) // len(c.kv_len))
    assert len(c.kv_len) * -(-rows // 16) * hkv > {128: 1216, 256: 800}[d]
    c.check(window, sinks)


@pytest.mark.parametrize("groups,hq,hkv,d,window", [
    ([(1500, [(1, 30)] * 70), (2500, [(2, 60)] * 50)], 8, 8, 128, 0),       # 960 tiles, room for 2,592 tokens: planned
    ([(2500, [(1, 30)] * 60)], 8, 8, 128, 0),                               # 480: one launch
    ([(700, [(3, 60)] * 60)], 8, 8, 256, 0), ([(900, [(3, 60)] * 60)], 8, 8, 256, 0),      # 480 tiles, up to 896 tokens of room and more
    ([(200, [(40, 60)] * 16)], 16, 8, 256, 0), ([(600, [(40, 60)] * 16)], 16, 8, 256, 0),  # 640 tiles of full rows
    ([(2200, [(1, 60)] * 100), (2000, [(1, 60)] * 100)], 8, 8, 64, 0),      # 1,600
    ([(4000, [(1, 60)] * 64)], 8, 8, 64, 0),                                # 512
    ([(5000, [(5, 60)] * 30)], 40, 8, 128, 2048),                           # by the window
])
def test_attend_on_both_sides_of_short(dev, groups, hq, hkv, d, window):
    """Against the layer's attention, as the large batches."""
    groups = [(p // 32 * 32, m) for p, m in groups]
    c = Branches(dev, groups, [], hq, hkv, d, 32, seed=hq + d, quick=True).upload()
    c.batch[2] = ints(np.maximum(c.table, 0), dev)
    q = c.q.to(dev)
    got = R.draft_branch_attend(q, *c.cache, *c.batch, window=window, sinks=4)
    want = L.draft_layer_attend(q, *c.cache, *c.batch[:3], window=window, sinks=4)
    assert all(torch.equal(a, b) for a, b in zip(got, R.draft_branch_attend(q, *c.cache, *c.batch, window=window, sinks=4)))
    assert float((got[1] - want[1]).abs().max()) < 1e-4
    assert float((got[0].float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())


@pytest.mark.parametrize("wide", [False, True])
def test_attend_is_the_layers(dev, wide):
    """Where the rows name one prefix's pages, draft_layer_attend of the same batch says the same."""
    c = Branches(dev, [(640, [(3, 50), (9, 70), (1, 1)]), (128, [(2, 30)] * 6)], [(4, 100)], 10, 2, 128, 64, seed=1, wide=wide)
    out, lse = c.check()
    want, lwant = L.draft_layer_attend(c.q.to(dev), *c.cache, *c.batch[:3])
    assert float((lse - lwant).abs().max()) < 1e-4 and float((out.float() - want.float()).abs().max()) < 0.02


@pytest.mark.parametrize("groups,loose,hq,hkv,d,window", [
    ([(20000, [(9, 60), (5, 40), (9, 10), (0, 5)]), (12000, [(9, 60)] * 4)], [], 40, 8, 128, 0),       # runs that hold several tiles
    ([(30000, [(100, 100), (70, 300)])], [], 64, 64, 64, 0),                                         # long runs, shares that are not even
    ([(3000, [(150 - i, 150) for i in range(12)])], [(200, 700)], 40, 8, 128, 0),                    # members with their prefix in them
    ([(700, [(1, 20 + i) for i in range(150)]), (2400, [(1, 9), (3, 90)] * 75)], [(2, 900)] * 9, 8, 2, 128, 0),      # many sequences
    ([(40 * i + 30, [(2, 3 + i)] * 2) for i in range(90)], [(1, 5)], 4, 2, 64, 0),                   # many groups
    ([(3000, [(4, 100)] * 20)], [(4, 2500)], 16, 2, 256, 0),
    ([(9000, [(4, 300)] * 12)], [(4, 5000)] * 2, 16, 2, 256, 2048),
    ([(2500, [(1, 3000 + i) for i in range(20)])], [], 8, 1, 64, 0),                                 # few rows over many tokens of their own
    ([(2500, [(1, 3000 + i) for i in range(20)])], [], 6, 3, 128, 3500),
    ([(60000, [(1, 1)])], [], 1, 1, 128, 0),
])
def test_attend_of_large_batches_is_the_layers(dev, groups, loose, hq, hkv, d, window):
    """Both attend to the same values: a difference is their rounding to bf16, of what is up to the largest of them."""
    c = Branches(dev, groups, loose, hq, hkv, d, 64, seed=hq + d, quick=True, wide=True).upload()
    c.table[c.table < 0] = 0      # a member's entry for the prefix's last page: the layer's call reads its own
    for g, (prefix, m) in enumerate(groups):
        for i in range(1, len(m)):
            s, j = int(c.group_start[g]) + i, prefix // 64
            if prefix % 64 and j < c.max_pages:      # the same tokens there
                a, b = c.table[int(c.group_start[g]), j], c.table[s, j]
                for x, byte in zip(c.cache[:2], (OL.key_byte, OL.value_byte)):
                    at = torch.tensor([byte(t, e, d) for t in range(prefix % 64) for e in range(d)], device=dev)
                    flat = x.view(x.shape[0], hkv, -1)
                    flat[int(b)][:, at] = flat[int(a)][:, at]
                for x in c.cache[2:]:
                    x[int(b)] = x[int(a)]
    c.batch[2] = ints(c.table, dev)
    q = c.q.to(dev)
    got = R.draft_branch_attend(q, *c.cache, *c.batch, window=window, sinks=4)
    want = L.draft_layer_attend(q, *c.cache, *c.batch[:3], window=window, sinks=4)
    again = R.draft_branch_attend(q, *c.cache, *c.batch, window=window, sinks=4)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert float((got[1] - want[1]).abs().max()) < 1e-4
    assert float((got[0].float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())


@pytest.mark.parametrize("wide", [False, True])
def test_attend_leaves_other_rows_alone(dev, wide):
    """Rows behind the last sequence, and a row stride."""
    c = Branches(dev, [(100, [(2, 20), (0, 3), (3, 9)])], [(1, 40)], 4, 2, 64, 32, seed=2, wide=wide)
    q = torch.zeros((c.rows + 5, 7, 64), dtype=torch.bfloat16, device=dev)[:, :4]
    q[:c.rows] = c.q.to(dev)
    out, lse = torch.full((c.rows + 5, 4, 64), 7.0, dtype=torch.bfloat16, device=dev), torch.full((c.rows + 5, 4), 7.0, device=dev)
    c.check(q=q, out=out, lse=lse)
    assert bool((out[c.rows:] == 7).all()) and bool((lse[c.rows:] == 7).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("new", [1, 30])
def test_attend_missing_pages_and_the_tables_end(dev, new, wide):
    c = Branches(dev, [(300, [(new, new + 40), (new, new + 10)])], [(new, 200)], 4, 1, 64, 32, seed=3, wide=wide)
    c.table[0, 3], c.table[1, 9], c.table[2, 2] = -1, 1 << 30, len(c.codes[0])
    c.check()
    for window, sinks in ((0, 0), (50, 3)):
        Branches(dev, [(300, [(new, new + 40), (new, new + 10)])], [(new, 400)], 4, 1, 64, 32, seed=4, max_pages=10).check(window, sinks)
        Branches(dev, [(2000, [(new, new + 200), (new, new + 60)])], [(new, 2300)], 4, 1, 64, 32, seed=4, max_pages=65).check(window, sinks)


@pytest.mark.parametrize("wide", [False, True])
def test_attend_of_values_that_are_no_numbers(dev, wide):
    """A page whose scale is none makes the rows that see it NaN, a query its own row; no others."""
    for new in (1, 30):
        c = Branches(dev, [(100, [(new, new + 10), (new, new + 40)]), (64, [(new, new), (new, new + 5)])], [], 4, 2, 64, 32, seed=5, wide=wide)
        c.scales[0][c.table[0, 1], 0] = np.nan          # the first group's prefix, the first kv head
        c.scales[1][c.table[3, 2 + (new + 4) // 32], 1] = np.inf      # a sequence's own last page, the second
        c.upload()
        q = c.q.to(dev)
        q[c.q_start[2], 0, 3] = float("inf")
        out, lse = R.draft_branch_attend(q, *c.cache, *c.batch)
        bad = torch.isnan(lse).cpu().numpy()
        want = np.zeros_like(bad)
        want[:c.q_start[2], :2] = True
        sees = np.arange(c.rows) >= c.q_start[3] + max(0, new - 1 - (new + 4) % 32)
        want[:, 2:] |= (sees & (np.arange(c.rows) >= c.q_start[3]))[:, None]
        want[c.q_start[2], 0] = True
        assert np.array_equal(bad, want) and np.array_equal(torch.isnan(out.float()).any(-1).cpu().numpy(), want)


@pytest.mark.parametrize("wide", [False, True])
def test_attend_groups_that_no_caller_should_have(dev, wide):
    """Row starts, groups and lengths that do not fit each other fault nothing and touch no row outside."""
    c = Branches(dev, [(100, [(3, 20), (3, 9)]), (64, [(2, 9)])], [(1, 40)], 4, 2, 64, 32, seed=6, wide=wide).upload()
    rng = np.random.default_rng(7)
    for t in range(12):
        start = ints(rng.integers(-5, 20, 5), dev)
        groups, prefix = ints(rng.integers(-3, 8, 3), dev), ints(rng.integers(-100, 1 << 30, 2), dev)
        out = torch.full((c.rows + 64, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
        R.draft_branch_attend(c.q.to(dev), *c.cache, start, c.batch[1] * (t % 3) - 9, c.batch[2], groups, prefix, window=t % 2 * 40, out=out[:c.rows])
        torch.cuda.synchronize()
        assert bool((out[c.rows:] == 7).all())


@pytest.mark.parametrize("wide", [False, True])
def test_attend_repeats_to_the_bit_on_another_stream_and_in_graphs(dev, wide):
    """Graphs that share one workspace, replayed in turn with eager calls between."""
    cases = [Branches(dev, [(900, [(1, 30)] * 9)], [(1, 50)], 10, 2, 128, 64, seed=8, wide=wide).upload(),
             Branches(dev, [(300, [(20, 60), (50, 50)])], [], 8, 2, 64, 32, seed=9, wide=wide).upload(),
             Branches(dev, [(300, [(1, 60)] * 70)], [], 8, 2, 64, 32, seed=9, wide=wide).upload()]
    ws = torch.full((max(R.draft_branch_attend_workspace_bytes(c.rows, len(c.kv_len), c.hq, c.hkv, c.d) for c in cases),), 255, dtype=torch.uint8, device=dev)
    graphs = []
    for c in cases:
        q = c.q.to(dev)
        want = R.draft_branch_attend(q, *c.cache, *c.batch)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = R.draft_branch_attend(q, *c.cache, *c.batch, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        outs = [torch.empty_like(t) for t in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            R.draft_branch_attend(q, *c.cache, *c.batch, out=outs[0], lse=outs[1], workspace=ws)
        graphs.append((graph, outs, want, q, c))
    for i in range(3):
        for graph, outs, want, q, c in graphs:
            for t in outs:
                t.fill_(3)
            ws.fill_(i * 100)
            graph.replay()
            eager = R.draft_branch_attend(q, *c.cache, *c.batch, workspace=ws)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(outs, want, eager))


def test_fork_then_attend(dev):
    """As they are used: prompts, their branches, a step of each branch over the shared pages, and the pool drawn together."""
    hq, hkv, d, page, n_pages = 10, 2, 128, 64, 80
    rng = np.random.default_rng(10)
    cache = L.DraftCache(n_pages, hkv, d, page, device=dev)
    lens = [300, 128, 77]
    table = np.full((3, 8), -1, np.int32)
    uses = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    none = torch.full((3,), -1, dtype=torch.int32, device=dev)
    zero = torch.zeros(3, dtype=torch.int32, device=dev)
    table, uses, status = cache.fork(uses, ints(table, dev), zero, none, ints(lens, dev))
    assert status.tolist() == [n_pages - sum(-(-n // page) for n in lens), 0]

    def made(rows):
        return [torch.from_numpy(rng.standard_normal((rows, h, d)).astype(np.float32)).to(torch.bfloat16).to(dev) for h in (hq, hkv, hkv)]

    q_start, kv_len = ints(np.concatenate([[0], np.cumsum(lens)]), dev), ints(lens, dev)
    q, k, v = made(sum(lens))
    cache.append(q, k, v, None, q_start, kv_len, table)
    parents = [0, 0, 0, 0, 2, 2]                     # the second ends
    branch_len = torch.tensor([lens[p] for p in parents], dtype=torch.int32, device=dev)
    more, counts, status = cache.fork(uses, table, kv_len, ints(parents, dev), branch_len + 3)
    assert int(status[1]) == 0 and int((counts > 0).sum()) == 4 + 4 + 1 + 2       # shared whole pages, and each branch's own
    groups, prefix = ints([0, 4, 6], dev), ints([300 // page * page, 77 // page * page], dev)
    for draw_together in (False, True):
        if draw_together:
            more, counts, status = cache.compact(counts, more)
            assert int(status[0]) == 11 and not bool((counts[11:] != 0).any())
        for step in range(3):
            length = branch_len + step + 1
            one = ints(list(range(7)), dev)
            q, k, v = made(6)
            cache.append(q, k, v, None, one, length, more)
            got = cache.attend_branches(q, one, length, more, groups, prefix)
            want = cache.attend(q, one, length, more)
            assert float((got[1] - want[1]).abs().max()) < 1e-4
            assert float((got[0].float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())
        first = cache.read(ints([0] + list(np.cumsum(branch_len.tolist())), dev), branch_len, more, int(branch_len.sum()))
        own_ = cache.read(q_start, kv_len, table, sum(lens)) if not draw_together else own_
        at = 0
        for p, n in zip(parents, branch_len.tolist()):     # every branch still has its parent's whole pages as they were
            whole = n // page * page
            lo = sum(lens[:p])
            assert all(torch.equal(a[at:at + whole], b[lo:lo + whole]) for a, b in zip(first, own_))
            at += n


# ---------------------------------------------------------- log probabilities
def rows_of(rng, m, n, kind):
    x = rng.standard_normal((m, n)).astype(np.float32) * 2
    if kind == "kept":
        x[rng.random((m, n)) > min(1.0, 30.0 / n)] = -np.inf
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "few values":
        x = np.rint(x)
    elif kind == "rising":
        x = np.sort(x, axis=1)
    elif kind == "falling":
        x = -np.sort(x, axis=1)
    elif kind == "peaked":
        x[np.arange(m), rng.integers(0, n, m)] = 40.0
    elif kind == "far":
        x = x * 60 - 5000
    elif kind == "lowest":
        x[:, ::3] = -3.3895313892515355e38      # bf16's lowest
    return x


def check_logprobs(dev, x, tokens, top, scale=1.0, scales=None, gap=0, dtype=None, **kw):
    m, n = x.shape
    dtype = dtype or torch.bfloat16
    wide = torch.full((m, n + gap), 99.0, dtype=dtype, device=dev)
    wide[:, :n] = torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(dev)
    x = wide[:, :n].float().cpu().numpy()
    given = None if scales is None else torch.from_numpy(np.asarray(scales, np.float32)).to(dev)
    got = R.draft_branch_logprobs(wide[:, :n], ints(tokens, dev), top=top, scale=scale, scales=given, **kw)
    torch.cuda.synchronize()
    factor = np.full(m, np.float32(scale)) * (np.ones(m, np.float32) if scales is None else np.asarray(scales, np.float32))
    want = O.logprobs(x, tokens, top, factor)
    logprob, top_id, top_logprob, lse, entropy = (t.cpu().numpy() for t in got)
    assert np.array_equal(top_id, want["top_id"])
    for name, t in (("logprob", logprob), ("top_logprob", top_logprob), ("lse", lse), ("entropy", entropy)):
        w = want[name]
        assert np.array_equal(np.isnan(t), np.isnan(w)) and np.array_equal(np.isneginf(t), np.isneginf(w)), name
    A = (n / 2048 + 3 * (20 + 256)) * U
    far, far2, peak = want["far"], want["far2"], want["max"]
    with np.errstate(invalid="ignore"):
        lnl = want["lse"] - peak
        ln_err = 4 * U * far + 2.0 ** -22 + A + 2 * U * np.abs(lnl)
        lims = {"lse": ln_err + U * np.abs(peak) + U * np.abs(want["lse"]),
                "entropy": ln_err + (2 * (2.0 ** -22 + A) + 8 * U) * far + 4 * U * far2 + U * want["entropy"]}
        for name in ("logprob", "top_logprob"):
            lims[name] = ln_err[:, None] + 3 * U * np.abs(want[name] + lnl[:, None]) + U * np.abs(want[name])
        for name, t in (("logprob", logprob), ("top_logprob", top_logprob), ("lse", lse), ("entropy", entropy)):
            fine = np.isfinite(want[name])
            err = np.abs(t.astype(np.float64) - want[name])
            assert np.all(err[fine] <= lims[name][fine]), (name, (err - lims[name])[fine].max())
    return got


KINDS = ["plain", "kept", "equal", "few values", "rising", "falling", "peaked", "far", "lowest"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,top,n_tok,gap", [(1, 1, 1, 1, 0), (3, 5, 8, 2, 3), (2, 2047, 64, 1, 1), (1, 9001, 20, 3, 0), (5, 30011, 64, 2, 7),
                                               (600, 4099, 8, 1, 0)])
def test_logprobs(dev, kind, m, n, top, n_tok, gap):
    rng = np.random.default_rng(n + top)
    x = rows_of(rng, m, n, kind)
    tokens = rng.integers(-1, n + 1, (m, n_tok))
    for dtype in (torch.bfloat16, torch.float32):
        check_logprobs(dev, x, tokens, top, scale=0.7, gap=gap, dtype=dtype)


LONG = [(kind, *sizes) for kind in ("plain", "few values", "rising", "falling", "equal", "peaked", "kept")
        for sizes in ((2, 140001, 64, 3), (3, 124160, 20, 0), (1, 1200007, 64, 0))] + [(kind, 1030, 20011, 20, 1) for kind in ("plain", "rising")]


@pytest.mark.parametrize("kind,m,n,top,gap", LONG)
def test_logprobs_of_long_rows(dev, kind, m, n, top, gap):
    """Rows of many steps: bounds that are raised on the way, more elements above them than are put down."""
    rng = np.random.default_rng(n + top + m)
    x = rows_of(rng, m, n, kind)
    for dtype in (torch.bfloat16, torch.float32):
        check_logprobs(dev, x, rng.integers(0, n, (m, 1)), top, gap=gap, dtype=dtype)


def test_logprobs_alternatives_at_the_edges(dev):
    """The best stand before the first 16 bytes' boundary and behind the last one; rows of few elements, at every alignment."""
    rng = np.random.default_rng(5)
    for n in (1, 2, 6, 7, 8, 9, 15, 16, 17, 23, 100, 4096, 4103, 9000):
        x = rows_of(rng, 9, n, "plain")
        x[:, 0] += 20
        x[:, -1] += 21
        for dtype in (torch.bfloat16, torch.float32):
            check_logprobs(dev, x, np.stack([np.zeros(9, np.int64), np.full(9, n - 1)], 1), 5, gap=1, dtype=dtype)


@pytest.mark.parametrize("m", [1, 9, 72, 128])
def test_logprobs_of_the_heads_row(dev, m):
    """The head's vocabulary shard, as many rows as it takes at once."""
    rng = np.random.default_rng(m)
    check_logprobs(dev, rows_of(rng, m, 124160, "plain"), rng.integers(0, 124160, (m, 1)), 8)


def test_logprobs_without_tokens_or_alternatives(dev):
    rng = np.random.default_rng(1)
    x = rows_of(rng, 4, 20000, "plain")
    check_logprobs(dev, x, np.zeros((4, 0), np.int32), 5)
    check_logprobs(dev, x, rng.integers(0, 20000, (4, 64)), 0)
    got = R.draft_branch_logprobs(torch.from_numpy(x).to(dev))
    assert got[0].shape == (4, 0) and got[1].shape == (4, 0) and bool(torch.isfinite(got[3]).all())
    none = R.draft_branch_logprobs(torch.empty((0, 100), device=dev), top=3)
    assert none[1].shape == (0, 3)


@pytest.mark.parametrize("m,n", [(4, 700), (4, 50000), (700, 700)])
def test_logprobs_of_rows_that_are_no_numbers(dev, m, n):
    """NaN, +inf, nothing but -inf, one element alone, factors that are none: each row for itself."""
    rng = np.random.default_rng(n)
    x = rows_of(rng, m, n, "plain")
    x[0, n // 2] = np.nan
    x[1] = -np.inf
    x[2, n - 1] = np.inf
    x[3] = -np.inf
    x[3, 17] = -4.0
    tokens = np.array([[3, n]] * (m - 1) + [[17, -5]])
    check_logprobs(dev, x, tokens, 4, dtype=torch.float32)
    check_logprobs(dev, x, tokens, 4)
    x[0, n // 2], x[2, n - 1] = 1.0, 2.0
    check_logprobs(dev, x, tokens, 4, scales=[0.5, 1.0, 2.0, 1e30] + [1.5] * (m - 4), scale=2.0)
    check_logprobs(dev, x, tokens, 4, scales=[0.0, -1.0, np.nan, np.inf] + [1.0] * (m - 4))
    x[0] = np.nan
    check_logprobs(dev, x, tokens, 4)


@pytest.mark.parametrize("top", [0, 4, 64])
@pytest.mark.parametrize("m,n", [(3, 700), (3, 9001), (700, 5000), (1030, 20011), (2, 124160)])
def test_logprobs_of_infinite_elements_before_the_first_bound(dev, m, n, top):
    """+inf in a row's first steps, in every wave, one and many: that row is NaN, its neighbours are not touched."""
    rng = np.random.default_rng(n + top)
    x = rows_of(rng, m, n, "plain")
    x[0, rng.integers(0, n, 40)] = np.inf
    x[m - 1] = np.inf
    for dtype in (torch.bfloat16, torch.float32):
        check_logprobs(dev, x, rng.integers(0, n, (m, 1)), top, gap=1, dtype=dtype)


@pytest.mark.parametrize("n", [5, 2047, 9001, 40000, 124160])
def test_logprobs_of_peaked_rows_are_small_and_right(dev, n):
    """One element far above the rest.  Its weight is 1 exactly and its distance 0, so what is left
    are the others' share W = sum e^d and D = sum e^d |d|, small numbers of their own:
      a lane       of k = n / (256 per) vectors of `per` elements moves its reference k times at most, the
                   lanes, waves and parts 9 times each: weights are e = (k + 18) 2^-22 + 4 u |d| off
      sum          adding to the peak's 1 loses u at most, and no more than what is added: min((k + per + 18) u, W)
      ln(sum)      that, e W and the logarithm's 2 u ln(sum): L
      entropy      L, and of D: e, the additions' (k + per + 54) u, 8 u
    A reference other than the peak leaves 2^-23 of its distance: 1e-7, where entropies here begin at 1e-12."""
    rng = np.random.default_rng(n)
    m = 24
    peak = rng.integers(0, n, m)
    peak[:2] = 0, n - 1
    for dtype, per in ((torch.bfloat16, 8), (torch.float32, 4)):
        x = rows_of(rng, m, n, "plain")
        x[np.arange(m), peak] = x.max(1) + np.linspace(1.0, 40.0, m)
        given = torch.from_numpy(x).to(dtype)
        x = given.double().numpy()
        d = x - x.max(1, keepdims=True)
        assert ((d == 0).sum(1) == 1).all()
        w = np.where(d < 0, np.exp(d), 0.0)
        W, D, D2 = w.sum(1), (w * -d).sum(1), (w * d * d).sum(1)
        k = n / (256 * per) + 1
        e = (k + 18) * 2.0 ** -22
        lnl, entropy = np.log1p(W), np.log1p(W) + D / (1 + W)
        L = np.minimum((k + per + 18) * U, W) + e * W + 4 * U * D + 2 * U * lnl
        lim = L + (e + (k + per + 62) * U) * D + 4 * U * D2 + (L + U) * D + U * entropy
        tokens = np.stack([peak, rng.integers(0, n, m)], 1)
        logprob, top_id, top_logprob, lse, got = (t.cpu().numpy() for t in R.draft_branch_logprobs(given.to(dev), ints(tokens, dev), top=3))
        assert np.array_equal(top_id[:, 0], peak)
        assert np.all(np.abs(got - entropy) <= lim), (np.abs(got - entropy) / lim).max()
        assert (lim < 0.2 * entropy)[W < 0.01].all() and entropy.min() < 1e-8 * n      # nothing else is as small
        for t in (logprob[:, 0], top_logprob[:, 0]):
            assert np.all(np.abs(t + lnl) <= L + U * lnl)
        assert np.all(np.abs(lse - x.max(1) - lnl) <= L + U * np.abs(lse))


def test_logprobs_of_the_largest_factors(dev):
    """Up to ln 2 times fp32's largest number a factor is one; beyond, every row is NaN, one without an element too."""
    rng = np.random.default_rng(6)
    x = rows_of(rng, 4, 5000, "plain") * np.float32(2.0 ** -127)
    x[3] = -np.inf
    tokens = rng.integers(0, 5000, (4, 2))
    for dtype in (torch.bfloat16, torch.float32):
        check_logprobs(dev, x, tokens, 4, scales=[1e38, 2.3e38, 2.35e38, 2.35e38], dtype=dtype)
        given = torch.from_numpy(x).to(dtype).to(dev)
        for f in (2.37e38, 3.0e38, 3.4028234e38):
            got = R.draft_branch_logprobs(given, ints(tokens, dev), top=4, scales=torch.full((4,), f, device=dev))
            assert all(bool(torch.isnan(got[i]).all()) for i in (0, 2, 3, 4)) and bool((got[1] == -1).all())


def test_logprobs_of_differences_past_the_largest_number(dev):
    """They are infinite: the element weighs nothing, though f would bring it near."""
    x = torch.full((2, 3000), -3e38)
    x[:, 7], x[:, 2900], x[1, 5] = 3e38, 2.9e38, 0.0
    logprob, top_id, top_logprob, lse, entropy = (t.double().cpu() for t in R.draft_branch_logprobs(
        x.to(dev), ints([[7, 2900, 5, 0]] * 2, dev), top=4, scales=torch.full((2,), 1e-37, device=dev)))
    z = torch.where(x > -1e38, x.double() * float(np.float32(1e-37)), -torch.inf)
    want = torch.log_softmax(z, 1)
    assert torch.equal(torch.isinf(logprob), torch.isinf(want[:, [7, 2900, 5, 0]])) and not torch.isnan(logprob).any()
    fine = torch.isfinite(logprob)
    assert float((logprob - want[:, [7, 2900, 5, 0]])[fine].abs().max()) < 2e-5      # 30 of z: u |z| and a few 2^-22
    assert float((lse - torch.logsumexp(z, 1)).abs().max()) < 2e-5
    assert float((entropy + torch.special.xlogy(want.exp(), want.exp()).sum(1)).abs().max()) < 2e-5
    assert top_id[0].tolist() == [7, 2900, 0, 1] and top_id[1].tolist() == [7, 2900, 5, 0] and bool(torch.isneginf(top_logprob[0, 2:]).all())


def test_logprobs_of_bits_and_shards(dev):
    """int16 rows are bf16 bits; two shards join by their lse."""
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rows_of(rng, 7, 6000, "plain")).to(torch.bfloat16).to(dev)
    tokens = ints(rng.integers(0, 6000, (7, 2)), dev)
    whole = R.draft_branch_logprobs(x, tokens, top=9)
    bits = R.draft_branch_logprobs(x.view(torch.int16), tokens, top=9)
    assert all(torch.equal(a, b) for a, b in zip(whole, bits))
    parts = [R.draft_branch_logprobs(x[:, a:b], tokens - a, top=9) for a, b in ((0, 2500), (2500, 6000))]
    lses = torch.stack([p[3] for p in parts]).double()
    lse = torch.logsumexp(lses, 0)
    entropy = lse - sum(torch.exp(p[3].double() - lse) * (p[3] - p[4]).double() for p in parts)
    logprob = torch.maximum(*(p[0].double() + (p[3].double() - lse)[:, None] for p in parts))
    for a, b in ((lse, whole[3]), (entropy, whole[4]), (logprob, whole[0])):
        assert float((a - b).abs().max()) < 1e-5


def test_logprobs_repeat_to_the_bit_on_another_stream_and_in_a_graph(dev):
    rng = np.random.default_rng(3)
    for m, n in ((1, 124160), (40, 9001), (900, 3001)):
        x = torch.from_numpy(rows_of(rng, m, n, "few values")).to(torch.bfloat16).to(dev)
        tokens = ints(rng.integers(0, n, (m, 1)), dev)
        want = R.draft_branch_logprobs(x, tokens, top=20)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = R.draft_branch_logprobs(x, tokens, top=20, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ws = torch.full((R.draft_branch_logprobs_workspace_bytes(m, n, 20),), 255, dtype=torch.uint8, device=dev)
        names = ("logprob", "top_id", "top_logprob", "lse", "entropy")
        outs = {k: torch.empty_like(t) for k, t in zip(names, want)}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            R.draft_branch_logprobs(x, tokens, top=20, workspace=ws, **outs)
        for i in range(3):
            for t in outs.values():
                t.fill_(3)
            ws.fill_(i)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[k], t) for k, t in zip(names, want))


def test_head_scores_its_tokens(dev):
    """The head's own call: its row's log probabilities, for a full and a top-k row."""
    from bit_quantized_lm_amd import workload
    n, k, m = 4000, 1024, 5
    head = B.DraftHead.from_weight(workload.gen_weight(n, k, seed=3), device=dev)
    x = torch.from_numpy(workload.gen_x(m, k, seed=4).view(np.int16)).to(dev)
    for topk_only in (False, True):
        first = head.logits_row(x, topk_only=topk_only)
        tokens = first["out_id"][:, None].contiguous()
        got = head.logprobs(x, tokens, top=3, scale=0.8, topk_only=topk_only)
        assert torch.equal(got["row"], first["row"]) and torch.equal(got["top_id"][:, 0], got["top_id"][:, 0].clamp(0, n - 1))
        want = O.logprobs(first["row"].view(torch.bfloat16).double().cpu().numpy(), tokens.cpu().numpy(), 3, np.full(m, np.float32(0.8)))
        assert np.array_equal(got["top_id"].cpu().numpy(), want["top_id"])
        assert np.abs(got["logprob"].cpu().numpy() - want["logprob"]).max() < 1e-4 and np.abs(got["entropy"].cpu().numpy() - want["entropy"]).max() < 1e-4


def test_head_on_another_stream(dev):
    """Memory that the current stream is still reading is not written by a call on another one, and the results are those of the current one."""
    from bit_quantized_lm_amd import workload
    n, k, m = 4000, 1024, 5
    head = B.DraftHead.from_weight(workload.gen_weight(n, k, seed=3), device=dev)
    x = torch.from_numpy(workload.gen_x(m, k, seed=4).view(np.int16)).to(dev)
    tokens = ints(np.arange(m)[:, None], dev)
    side = torch.cuda.Stream()
    calls = [lambda s: head(x, stream=s), lambda s: head.logits_row(x, stream=s), lambda s: head.logits_row_staged(x, stream=s),
             lambda s: head.staged(x, stream=s), lambda s: head.logprobs(x, tokens, top=3, scale=0.8, stream=s)]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        for s in (side, side.cuda_stream):
            # blocks of the sizes that the call takes, freed while a copy of them waits
            busy = [torch.full_like(t, 7) for t in want.values()] + [torch.full((1 << 16,), 7, dtype=torch.uint8, device=dev)]
            copies = [torch.empty_like(t) for t in busy]
            torch.cuda.synchronize()
            torch.cuda._sleep(4_000_000)
            for a, b in zip(copies, busy):
                a.copy_(b)
            del busy, b
            got = call(s)
            side.synchronize()
            for name, t in want.items():
                assert torch.equal(got[name], t), name
            torch.cuda.synchronize()
            assert all(bool((t == 7).all()) for t in copies)
