"""The operators on several branches on the CPU: exported names, every refusal
(all arguments are checked before any HIP call, so none needs a GPU), sizes of
workspaces."""
import ctypes

import pytest

from bit_quantized_lm_amd import _binding as B
from bit_quantized_lm_amd import _branch as R


@pytest.fixture(scope="module")
def lib():
    try:
        return R._load()
    except FileNotFoundError:
        import __graft_entry__
        __graft_entry__.build()
        return R._load()


def test_every_header_function_is_exported_and_bound(lib):
    names = R.branch_header_functions()
    assert len(names) == len(set(names)) >= 5
    for name in names:
        assert hasattr(lib, name) and callable(getattr(R, name)), name


def test_package_names():
    import bit_quantized_lm_amd as pkg
    for name in pkg._BRANCH_NAMES:
        assert getattr(pkg, name) is getattr(R, name) and name in pkg.__all__
    with open(R._HEADER) as f:
        text = f.read()
    assert f"#define DB_MAX_TOP {R.MAX_TOP}\n" in text and "#define DB_BF16 0\n" in text and "#define DB_FP32 1\n" in text


# --------------------------------------------------------------- refusals
P = 1 << 20       # stands for device addresses: nothing is read before the checks are done
FAR = 1 << 24     # and this one for buffers that do not overlap those

FORK = dict(kc=P, vc=P, ks=P, vs=P, n_pages=9, page=64, hkv=2, D=128, uses=P, table=P, kv_len=P, n_seq=3, parents=P, need=P, n_new=5,
            max_pages=10, uses_out=FAR, table_out=2 * FAR, status=3 * FAR, workspace=P, bytes=1 << 40, stream=None)
COMPACT = dict(kc=P, vc=P, ks=P, vs=P, n_pages=9, page=64, hkv=2, D=128, uses=P, table=P, n_rows=3, max_pages=10, uses_out=FAR,
               table_out=2 * FAR, status=3 * FAR, workspace=P, bytes=1 << 40, stream=None)
LOGPROBS = dict(x=P, type=0, ld=1000, M=3, N=1000, scale=1.0, scales=None, tokens=P, n_tok=1, top=8, logprob=P, lse=P, entropy=P, top_id=P,
                top_logprob=P, workspace=P, bytes=1 << 40, stream=None)

ATTEND = dict(q=P, ldq=1024, kc=P, vc=P, ks=P, vs=P, n_pages=9, page=64, q_start=P, kv_len=P, table=P, n_seq=3, max_pages=10, group_start=P,
              prefix_len=P, n_groups=2, T=5, hq=8, hkv=2, D=128, scale=0.1, window=0, sinks=0, out=P, lse=P, workspace=P, bytes=1 << 40,
              stream=None)

PAGES = [(dict(D=96), B.DH_EUNSUP), (dict(hkv=0), B.DH_ESHAPE), (dict(hkv=257), B.DH_ESHAPE), (dict(kc=None), B.DH_EINVAL),
         (dict(vc=None), B.DH_EINVAL), (dict(ks=None), B.DH_EINVAL), (dict(vs=None), B.DH_EINVAL), (dict(kc=P + 8), B.DH_EINVAL),
         (dict(vs=P + 2), B.DH_EINVAL), (dict(page=48), B.DH_EUNSUP), (dict(n_pages=0), B.DH_ESHAPE), (dict(n_pages=(1 << 24) + 1), B.DH_ESHAPE),
         (dict(max_pages=0), B.DH_ESHAPE), (dict(max_pages=1 << 24), B.DH_ESHAPE), (dict(uses=None), B.DH_EINVAL), (dict(uses=P + 1), B.DH_EINVAL),
         (dict(table=None), B.DH_EINVAL), (dict(table=P + 2), B.DH_EINVAL), (dict(uses_out=None), B.DH_EINVAL), (dict(table_out=None), B.DH_EINVAL),
         (dict(status=None), B.DH_EINVAL), (dict(status=FAR + 2), B.DH_EINVAL), (dict(uses_out=P), B.DH_EINVAL), (dict(uses_out=P + 32), B.DH_EINVAL),
         (dict(table_out=P), B.DH_EINVAL), (dict(table_out=P - 4), B.DH_EINVAL), (dict(status=P + 4), B.DH_EINVAL), (dict(workspace=None), B.DH_EINVAL),
         (dict(workspace=P + 4), B.DH_EINVAL), (dict(bytes=10), B.DH_EINVAL),
         (dict(status=FAR), B.DH_EINVAL), (dict(status=2 * FAR + 116), B.DH_EINVAL), (dict(table_out=FAR + 32), B.DH_EINVAL)]


def _refused(lib, f, args, change, want, who):
    rc = f(*{**args, **change}.values())
    assert rc == want, (change, rc, lib.draft_head_last_error())
    assert who in lib.draft_head_last_error()


@pytest.mark.parametrize("change,want", PAGES + [
    (dict(n_seq=0), B.DH_ESHAPE), (dict(n_seq=4097), B.DH_ESHAPE), (dict(n_new=0), B.DH_ESHAPE), (dict(n_new=4097), B.DH_ESHAPE),
    (dict(kv_len=None), B.DH_EINVAL), (dict(parents=None), B.DH_EINVAL), (dict(need=None), B.DH_EINVAL), (dict(need=P + 1), B.DH_EINVAL),
    (dict(kv_len=FAR), B.DH_EINVAL), (dict(parents=2 * FAR + 196), B.DH_EINVAL), (dict(need=3 * FAR - 16), B.DH_EINVAL),
    (dict(n_new=128, max_pages=1 << 24), B.DH_ESHAPE), (dict(n_new=4096, max_pages=1 << 19), B.DH_ESHAPE)])
def test_fork_refuses(lib, change, want):
    _refused(lib, lib.draft_branch_fork, FORK, change, want, b"fork")


@pytest.mark.parametrize("change", [
    dict(status=FAR), dict(status=FAR + 32), dict(status=2 * FAR + 196), dict(table_out=FAR), dict(uses_out=3 * FAR - 32), dict(uses_out=P),
    dict(table_out=P - 196), dict(kv_len=FAR - 8), dict(parents=2 * FAR + 196), dict(need=3 * FAR + 4)])
def test_fork_refuses_what_overlaps(lib, change):
    _refused(lib, lib.draft_branch_fork, FORK, change, B.DH_EINVAL, b"overlap")


# buffers that follow each other without a gap, in units of 1 MiB: n_pages 64 of 64 KiB make a cache of 4 MiB codes twice
APART = {name: (i + 16) << 20 for i, name in enumerate(("uses", "table", "kv_len", "parents", "need", "uses_out", "table_out", "status", "workspace", "ks", "vs"))}
APART.update(kc=64 << 20, vc=68 << 20, n_pages=64, page=256, hkv=2, D=128)
SIZES = dict(uses=256, table=120, kv_len=12, parents=20, need=20, uses_out=256, table_out=0, status=8, ks=512, vs=512, kc=4 << 20, vc=4 << 20)


@pytest.mark.parametrize("f,args", [("draft_branch_fork", FORK), ("draft_branch_compact", COMPACT)])
def test_pages_refuse_what_overlaps_the_workspace_or_the_cache(lib, f, args):
    """The kernels write pages and workspace while they go by counts, tables and what they left in the workspace."""
    apart = {k: v for k, v in APART.items() if k in args}
    written = ("workspace", "kc", "vc", "ks", "vs")
    for a in written:
        for b in set(apart) & set(SIZES):
            if a == b or {a, b} <= set(written[1:]):      # the cache's own four are the caller's to keep apart
                continue
            size = {**SIZES, "table_out": 4 * args["max_pages"] * args.get("n_new", args.get("n_rows"))}
            for at in {apart[a], apart[a] + size.get(a, 16) - 4, apart[a] - size[b] + 4}:      # of the workspace the first bytes at least
                change = {**apart, b: at // 16 * 16 if b in ("kc", "vc") else at}
                if change["workspace"] % 16 == 0:
                    _refused(lib, getattr(lib, f), args, change, B.DH_EINVAL, b"overlap")


def test_fork_takes_buffers_that_follow_each_other(lib):
    """Refused for the misaligned list alone, which is looked at last."""
    for change in (dict(), dict(workspace=APART["kc"] - 4096, bytes=4096), dict(uses_out=APART["kc"] - 256), dict(table_out=APART["kc"] + (8 << 20)),
                   dict(status=APART["uses"] + 256), dict(parents=APART["kv_len"] + 12, need=APART["kv_len"] + 33), dict(kv_len=APART["uses"])):
        rc = lib.draft_branch_fork(*{**FORK, **APART, "need": APART["need"] + 1, **change}.values())
        assert rc == B.DH_EINVAL and b"aligned" in lib.draft_head_last_error(), (change, lib.draft_head_last_error())


@pytest.mark.parametrize("change,want", PAGES + [(dict(n_rows=0), B.DH_ESHAPE), (dict(n_rows=4097), B.DH_ESHAPE)])
def test_compact_refuses(lib, change, want):
    _refused(lib, lib.draft_branch_compact, COMPACT, change, want, b"compact")


@pytest.mark.parametrize("change,want", [
    (dict(D=96), B.DH_EUNSUP), (dict(hkv=0), B.DH_ESHAPE), (dict(hq=7), B.DH_ESHAPE), (dict(hq=512), B.DH_ESHAPE), (dict(T=-1), B.DH_ESHAPE),
    (dict(T=1 << 23), B.DH_ESHAPE), (dict(n_seq=0), B.DH_ESHAPE), (dict(n_seq=4097), B.DH_ESHAPE), (dict(n_groups=0), B.DH_ESHAPE),
    (dict(n_groups=4), B.DH_ESHAPE), (dict(kc=None), B.DH_EINVAL), (dict(vc=P + 8), B.DH_EINVAL), (dict(ks=None), B.DH_EINVAL),
    (dict(q_start=None), B.DH_EINVAL), (dict(kv_len=P + 2), B.DH_EINVAL), (dict(table=None), B.DH_EINVAL), (dict(page=16), B.DH_EUNSUP),
    (dict(max_pages=0), B.DH_ESHAPE), (dict(max_pages=1 << 24), B.DH_ESHAPE), (dict(n_pages=0), B.DH_ESHAPE), (dict(group_start=None), B.DH_EINVAL),
    (dict(prefix_len=None), B.DH_EINVAL), (dict(prefix_len=P + 1), B.DH_EINVAL), (dict(group_start=P + 2), B.DH_EINVAL), (dict(scale=0.0), B.DH_EINVAL),
    (dict(scale=float("nan")), B.DH_EINVAL), (dict(window=-1), B.DH_EINVAL), (dict(sinks=-1), B.DH_EINVAL), (dict(q=None), B.DH_EINVAL),
    (dict(q=P + 8), B.DH_EINVAL), (dict(ldq=1028), B.DH_EINVAL), (dict(ldq=1016), B.DH_EINVAL), (dict(out=None), B.DH_EINVAL),
    (dict(out=P + 8), B.DH_EINVAL), (dict(lse=P + 2), B.DH_EINVAL), (dict(workspace=None), B.DH_EINVAL), (dict(workspace=P + 8), B.DH_EINVAL),
    (dict(bytes=1000), B.DH_EINVAL)])
def test_attend_refuses(lib, change, want):
    _refused(lib, lib.draft_branch_attend, ATTEND, change, want, b"attend")


def test_attend_refuses_what_overlaps(lib):
    """A second launch goes by what the first one left in the workspace, and by the row starts."""
    at = dict(q=1 << 30, kc=2 << 30, vc=3 << 30, ks=4 << 30, vs=5 << 30)
    names = ("q_start", "kv_len", "table", "group_start", "prefix_len", "out", "lse", "workspace")
    at.update({k: (6 << 30) + (i << 28) for i, k in enumerate(names)})
    size = dict(q_start=16, kv_len=12, table=120, group_start=12, prefix_len=8, out=5 * 8 * 128 * 2, lse=5 * 8 * 4, workspace=4096)
    for a in names[5:]:
        for b in names:
            for there in {at[a], at[a] + size[a] - 16, at[a] - size[b] + 16 & -16}:
                if a != b and there < at[a] + size[a] and there + size[b] > at[a]:
                    _refused(lib, lib.draft_branch_attend, ATTEND, {**at, b: there}, B.DH_EINVAL, b"overlap")


@pytest.mark.parametrize("hq,hkv,d", [(40, 8, 128), (7, 7, 256), (16, 1, 64), (16, 2, 256), (200, 200, 64), (256, 1, 128)])
def test_attend_takes_the_largest_batchs_workspace(lib, hq, hkv, d):
    """The size never falls as rows or sequences grow, and no smaller call asks for more."""
    import re
    rows, seqs = (0, 1, 2, 5, 16, 17, 64, 65, 500, 4096), (1, 2, 3, 8, 63, 64, 500)
    size = {(t, n): R.draft_branch_attend_workspace_bytes(t, n, hq, hkv, d) for t in rows for n in seqs}
    for (t, n), most in size.items():
        assert all(most >= other for (u, m), other in size.items() if u <= t and m <= n)
    for t in rows[1:]:
        for n in seqs:
            for g in {1, min(2, n), n // 2 or 1, n}:
                _refused(lib, lib.draft_branch_attend, ATTEND, dict(T=t, n_seq=n, n_groups=g, hq=hq, hkv=hkv, D=d, ldq=hq * d, bytes=16),
                         B.DH_EINVAL, b"attend")
                need = int(re.search(rb"below the (\d+) needed", lib.draft_head_last_error()).group(1))
                assert 16 < need <= size[t, n], (t, n, g)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), B.DH_ESHAPE), (dict(M=(1 << 22) + 1), B.DH_ESHAPE), (dict(N=0), B.DH_ESHAPE), (dict(N=(1 << 24) + 1), B.DH_ESHAPE),
    (dict(top=-1), B.DH_EUNSUP), (dict(top=65), B.DH_EUNSUP), (dict(n_tok=-1), B.DH_EUNSUP), (dict(n_tok=65), B.DH_EUNSUP),
    (dict(type=2), B.DH_EUNSUP), (dict(ld=999), B.DH_EINVAL), (dict(scale=0.0), B.DH_EINVAL), (dict(scale=-1.0), B.DH_EINVAL),
    (dict(scale=float("nan")), B.DH_EINVAL), (dict(scale=float("inf")), B.DH_EINVAL), (dict(x=None), B.DH_EINVAL), (dict(x=P + 1), B.DH_EINVAL),
    (dict(x=P + 2, type=1), B.DH_EINVAL), (dict(tokens=None), B.DH_EINVAL), (dict(logprob=None), B.DH_EINVAL), (dict(lse=None), B.DH_EINVAL),
    (dict(entropy=None), B.DH_EINVAL), (dict(top_id=None), B.DH_EINVAL), (dict(top_logprob=None), B.DH_EINVAL), (dict(scales=P + 2), B.DH_EINVAL),
    (dict(lse=P + 2), B.DH_EINVAL), (dict(N=100000, ld=100000, workspace=None), B.DH_EINVAL), (dict(N=100000, ld=100000, workspace=P + 8), B.DH_EINVAL),
    (dict(N=100000, ld=100000, bytes=100), B.DH_EINVAL)])
def test_logprobs_refuses(lib, change, want):
    _refused(lib, lib.draft_branch_logprobs, LOGPROBS, change, want, b"logprobs")


def test_no_rows_is_no_work(lib):
    assert lib.draft_branch_logprobs(*{**LOGPROBS, "M": 0, "x": None, "lse": None}.values()) == B.DH_OK
    assert lib.draft_branch_attend(*{**ATTEND, "T": 0, "q": None}.values()) == B.DH_OK


def test_workspace_bytes(lib):
    null = ctypes.POINTER(ctypes.c_size_t)()
    assert lib.draft_branch_pages_workspace_bytes(1, 1, null) == B.DH_EINVAL
    assert lib.draft_branch_logprobs_workspace_bytes(1, 1, 1, null) == B.DH_EINVAL
    for bad in ((0, 1), (1, 0), (1 << 25, 1), (1, 4097)):
        with pytest.raises(ValueError):
            R.draft_branch_pages_workspace_bytes(*bad)
    for bad in ((-1, 5, 0), (1, 0, 0), (1, 5, 65), (1, 5, -1)):
        with pytest.raises(ValueError):
            R.draft_branch_logprobs_workspace_bytes(*bad)
    assert R.draft_branch_logprobs_workspace_bytes(0, 5, 0) == 0


def test_workspace_of_the_largest_serves_smaller_ones(lib):
    """The sizes never fall, and no smaller call asks for more (what a call asks for
    is in its refusal of a workspace of no bytes)."""
    import re
    sizes = [(n, r, R.draft_branch_pages_workspace_bytes(n, r)) for n in (1, 7, 2048, 2049, 100000, 1 << 24) for r in (1, 5, 4096)]
    for n, r, size in sizes:
        assert all(size >= other for m, q, other in sizes if m <= n and q <= r)
        for f, args, name in ((lib.draft_branch_fork, FORK, "n_new"), (lib.draft_branch_compact, COMPACT, "n_rows")):
            far = {k: i << 40 for i, k in enumerate(("uses_out", "table_out", "status"), 1)}
            _refused(lib, f, args, {"n_pages": n, name: r, "bytes": 0, **far}, B.DH_EINVAL, b"below the")
            need = int(re.search(rb"below the (\d+) needed", lib.draft_head_last_error()).group(1))
            assert 0 < need <= size
    for most in (1, 3, 72, 128, 700, 1024, 5000):
        for top in (0, 1, 8, 20, 64):
            size = R.draft_branch_logprobs_workspace_bytes(most, 250000, top)
            for m in (1, 2, 3, 5, 17, 72, 100, 128, 511, 513, 700, 1023, 1024, 1025, 5000):
                for n in (1, 2047, 4096, 4097, 30000, 124160, 250000):
                    for k in (0, 1, 7, 20, 64):
                        if m > most or k > top:
                            continue
                        rc = lib.draft_branch_logprobs(*{**LOGPROBS, "M": m, "N": n, "ld": n, "top": k, "bytes": 0, "scale": 0.0}.values())
                        assert rc == B.DH_EINVAL
                        rc = lib.draft_branch_logprobs(*{**LOGPROBS, "M": m, "N": n, "ld": n, "top": k, "bytes": 0, "x": None}.values())
                        assert rc == B.DH_EINVAL
                        # parts beyond one ask for a workspace
                        if n > 4096 and m < 512:
                            _refused(lib, lib.draft_branch_logprobs, LOGPROBS, {"M": m, "N": n, "ld": n, "top": k, "bytes": 0}, B.DH_EINVAL, b"below the")
                            need = int(re.search(rb"below the (\d+) needed", lib.draft_head_last_error()).group(1))
                            assert 0 < need <= size, (most, top, m, n, k)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    c, s, i = torch.zeros((2, 1, 32, 64), dtype=torch.uint8), torch.ones((2, 1)), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        R.draft_branch_fork(c, c, s, s, i, table, i[:1], i, i)
    with pytest.raises(ValueError, match="parents"):
        R.draft_branch_fork(c, c, s, s, i, table, i[:1], i[0], i)
    with pytest.raises(ValueError):
        R.draft_branch_compact(c, c, s, s, i, table)
    with pytest.raises(ValueError):
        R.draft_branch_attend(torch.zeros((1, 1, 64), dtype=torch.bfloat16), c, c, s, s, i, i[:1], table, i, i[:1])
    with pytest.raises(ValueError):
        R.draft_branch_logprobs(torch.zeros((2, 5)), torch.zeros((2, 1), dtype=torch.int32))
