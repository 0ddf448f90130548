"""The draft layer's attention on the CPU: the rotary table against the float64
oracle, the stored byte order, and every refusal (all arguments are checked
before any HIP call, so none needs a GPU)."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

from bit_quantized_lm_amd import _binding as B
from bit_quantized_lm_amd import _layer as L
from oracle import layer as O


@pytest.fixture(scope="module")
def lib():
    try:
        return L._load()
    except FileNotFoundError:
        import __graft_entry__
        __graft_entry__.build()
        return L._load()


def test_every_header_function_is_exported_and_bound(lib):
    names = L.layer_header_functions()
    assert set(names) == {"draft_layer_rope_table", "draft_layer_append", "draft_layer_read", "draft_layer_workspace_bytes",
                          "draft_layer_attend"}
    for name in names:
        assert hasattr(lib, name) and callable(getattr(L, name)), name


def test_package_names():
    import bit_quantized_lm_amd as pkg
    for name in pkg._LAYER_NAMES:
        assert getattr(pkg, name) is getattr(L, name)


@pytest.mark.parametrize("kw", [
    dict(positions=1, rot=2),
    dict(positions=5000, rot=128),
    dict(positions=300, rot=64, base=500000.0, factor=8.0),
    dict(positions=9000, rot=128, base=10000.0, factor=16.0, original=4096),
    dict(positions=64, rot=256, base=1e6, factor=4.0, original=32768, beta_fast=16.0, beta_slow=2.0, mscale=1.25),
    dict(positions=40, rot=16, base=10000.0, factor=2.0, original=8),      # the ramp's ends fall together
])
def test_rope_table(lib, kw):
    got = L.draft_layer_rope_table(**kw)
    m = kw.get("mscale")
    if m is None:
        m = 0.1 * math.log(kw["factor"]) + 1.0 if kw.get("original", 0) > 0 else 1.0
    want = O.rope_table(**{**kw, "mscale": m})
    assert got.dtype == np.float32 and got.shape == want.shape
    # one rounding to fp32 (2^-24 relative), and double's own: the angle p f has relative error under 2^-50
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + m * kw["positions"] * 2.0 ** -49 + 1e-45)


def test_rope_scaling_kinds(lib):
    plain = L.draft_layer_rope_table(64, 128)
    slow = L.draft_layer_rope_table(256, 128, factor=4.0)
    assert np.allclose(slow[::4], plain, atol=1e-6)                        # positions interpolated
    yarn = L.draft_layer_rope_table(256, 128, factor=4.0, original=4096, mscale=1.0)
    wide = L.draft_layer_rope_table(256, 128)
    assert np.array_equal(yarn[:, 0], wide[:, 0])                          # the fastest pair keeps its frequency
    assert np.allclose(yarn[:, -1], slow[:, -1], atol=1e-7)                # the slowest is interpolated


@pytest.mark.parametrize("change", [dict(positions=0), dict(positions=2 ** 30 + 1), dict(rot=0), dict(rot=3), dict(rot=258),
                                    dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(factor=float("inf")),
                                    dict(original=-1), dict(beta_fast=0.0), dict(beta_slow=-1.0), dict(mscale=0.0)])
def test_rope_table_refuses(lib, change):
    a = {**dict(positions=4, rot=8, base=1e4, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0, mscale=1.0), **change}
    out = np.zeros(64, np.float32)
    rc = lib.draft_layer_rope_table(a["positions"], a["rot"], a["base"], a["factor"], a["original"], a["beta_fast"],
                                    a["beta_slow"], a["mscale"], out.ctypes.data)
    assert rc in (B.DH_EINVAL, B.DH_ESHAPE) and b"rope_table" in lib.draft_head_last_error()
    assert not out.any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 256])
def test_stored_order_is_a_permutation(d, page):
    t, e = np.meshgrid(np.arange(page), np.arange(d), indexing="ij")
    for byte_of in (O.key_byte, O.value_byte):
        assert np.array_equal(np.sort(byte_of(t, e, d).ravel()), np.arange(page * d))


# --------------------------------------------------------------- refusals
P = 4096          # stands for a device address: nothing is read before the checks are done

APPEND = dict(q=P, ldq=1024, k=P, ldk=256, v=P, ldv=256, rope=P, positions=640, rot=128, inter=0, kc=P, vc=P, ks=P, vs=P, n_pages=9,
              page=64, q_start=P, kv_len=P, table=P, n_seq=2, max_pages=10, T=5, hq=8, hkv=2, D=128, q_out=P, stream=None)
READ = dict(kc=P, vc=P, ks=P, vs=P, n_pages=9, page=64, q_start=P, kv_len=P, table=P, n_seq=2, max_pages=10, T=5, hkv=2, D=128,
            k_out=P, v_out=P, stream=None)
ATTEND = dict(q=P, ldq=1024, kc=P, vc=P, ks=P, vs=P, n_pages=9, page=64, q_start=P, kv_len=P, table=P, n_seq=2, max_pages=10, T=5,
              hq=8, hkv=2, D=128, scale=0.1, window=0, sinks=0, out=P, lse=P, workspace=P, bytes=1 << 40, stream=None)

COMMON = [(dict(D=96), B.DH_EUNSUP), (dict(D=0), B.DH_EUNSUP), (dict(hkv=0), B.DH_ESHAPE), (dict(T=-1), B.DH_ESHAPE),
          (dict(T=1 << 23), B.DH_ESHAPE), (dict(n_seq=0), B.DH_ESHAPE), (dict(n_seq=4097), B.DH_ESHAPE), (dict(kc=None), B.DH_EINVAL),
          (dict(vc=None), B.DH_EINVAL), (dict(ks=None), B.DH_EINVAL), (dict(vs=None), B.DH_EINVAL), (dict(q_start=None), B.DH_EINVAL),
          (dict(kv_len=None), B.DH_EINVAL), (dict(table=None), B.DH_EINVAL), (dict(kc=P + 8), B.DH_EINVAL), (dict(vc=P + 4), B.DH_EINVAL),
          (dict(ks=P + 2), B.DH_EINVAL), (dict(table=P + 1), B.DH_EINVAL), (dict(page=48), B.DH_EUNSUP), (dict(page=16), B.DH_EUNSUP),
          (dict(page=512), B.DH_EUNSUP), (dict(n_pages=0), B.DH_ESHAPE), (dict(max_pages=0), B.DH_ESHAPE),
          (dict(max_pages=1 << 24), B.DH_ESHAPE)]


def _refused(lib, f, args, change, want, who):
    rc = f(*{**args, **change}.values())
    assert rc == want, (change, rc, lib.draft_head_last_error())
    assert who in lib.draft_head_last_error()


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(hq=7), B.DH_ESHAPE), (dict(hq=1), B.DH_ESHAPE), (dict(hq=512), B.DH_ESHAPE), (dict(rot=8), B.DH_ESHAPE),
    (dict(rot=144), B.DH_ESHAPE), (dict(rot=-16), B.DH_ESHAPE), (dict(rope=None), B.DH_EINVAL), (dict(rope=P + 4), B.DH_EINVAL),
    (dict(positions=639), B.DH_ESHAPE), (dict(q_out=None), B.DH_EINVAL), (dict(q=None), B.DH_EINVAL), (dict(k=None), B.DH_EINVAL),
    (dict(v=None), B.DH_EINVAL), (dict(ldk=255), B.DH_EINVAL), (dict(ldk=248), B.DH_EINVAL), (dict(ldv=128), B.DH_EINVAL),
    (dict(ldq=1020), B.DH_EINVAL), (dict(ldq=512), B.DH_EINVAL), (dict(k=P + 2), B.DH_EINVAL), (dict(q_out=P + 8), B.DH_EINVAL),
    (dict(ldq=2048), B.DH_EINVAL)])       # q_out is q here, so q must have no gaps
def test_append_refuses(lib, change, want):
    _refused(lib, lib.draft_layer_append, APPEND, change, want, b"append")


@pytest.mark.parametrize("change,want", COMMON + [(dict(k_out=None), B.DH_EINVAL), (dict(v_out=P + 8), B.DH_EINVAL)])
def test_read_refuses(lib, change, want):
    _refused(lib, lib.draft_layer_read, READ, change, want, b"read")


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(hq=7), B.DH_ESHAPE), (dict(scale=0.0), B.DH_EINVAL), (dict(scale=-1.0), B.DH_EINVAL), (dict(scale=float("nan")), B.DH_EINVAL),
    (dict(scale=float("inf")), B.DH_EINVAL), (dict(window=-1), B.DH_EINVAL), (dict(sinks=-1), B.DH_EINVAL), (dict(q=None), B.DH_EINVAL),
    (dict(ldq=1028), B.DH_EINVAL), (dict(ldq=1016), B.DH_EINVAL), (dict(out=None), B.DH_EINVAL), (dict(out=P + 8), B.DH_EINVAL),
    (dict(lse=P + 2), B.DH_EINVAL), (dict(workspace=None), B.DH_EINVAL), (dict(workspace=P + 8), B.DH_EINVAL),
    (dict(bytes=1000), B.DH_EINVAL)])
def test_attend_refuses(lib, change, want):
    _refused(lib, lib.draft_layer_attend, ATTEND, change, want, b"attend")


def test_no_rows_is_no_work(lib):
    assert lib.draft_layer_append(*{**APPEND, "T": 0}.values()) == B.DH_OK
    assert lib.draft_layer_read(*{**READ, "T": 0}.values()) == B.DH_OK
    assert lib.draft_layer_attend(*{**ATTEND, "T": 0}.values()) == B.DH_OK


def test_workspace_bytes(lib):
    assert L.draft_layer_workspace_bytes(1, 1, 40, 8, 128) > 0
    assert L.draft_layer_workspace_bytes(0, 1, 8, 8, 64) > 0
    for bad in ((1, 1, 40, 8, 100), (1, 1, 40, 7, 128), (-1, 1, 8, 8, 64), (1, 0, 8, 8, 64)):
        with pytest.raises(ValueError):
            L.draft_layer_workspace_bytes(*bad)
    assert lib.draft_layer_workspace_bytes(1, 1, 8, 8, 64, ctypes.POINTER(ctypes.c_size_t)()) == B.DH_EINVAL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    c = torch.zeros((2, 1, 32, 64), dtype=torch.uint8)
    s = torch.ones((2, 1))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.draft_layer_read(c, c, s, s, i, i[:1], torch.zeros((1, 2), dtype=torch.int32), 0)
    with pytest.raises(ValueError):
        L.DraftCache(4, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        L.DraftCache(4, 2, 64, page=48, device="cpu")


def test_workspace_clears_its_counters_alone(lib, monkeypatch):
    """A new workspace costs the clearing of its counters, whatever its size."""
    torch = pytest.importorskip("torch")
    with open(L._HEADER) as f:
        assert f"#define DL_WORKSPACE_ZERO_BYTES {L.WORKSPACE_ZERO_BYTES} " in f.read()
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).fill_(255))
    ws = L.draft_layer_workspace(72, 8, 40, 8, 128, "cpu")
    assert ws.numel() == L.draft_layer_workspace_bytes(72, 8, 40, 8, 128) > 1 << 20
    assert not ws[:L.WORKSPACE_ZERO_BYTES].any() and bool((ws[L.WORKSPACE_ZERO_BYTES:] == 255).all())


@pytest.mark.parametrize("hq,hkv,d", [(40, 8, 128), (7, 7, 256), (16, 2, 256), (8, 1, 64), (56, 8, 64), (256, 1, 128), (200, 200, 64)])
def test_workspace_of_the_largest_batch_serves_smaller_ones(lib, hq, hkv, d):
    """The size never falls as rows or sequences grow."""
    rows = [0, 1, 2, 3, 4, 8, 12, 13, 16, 17, 32, 63, 64, 65, 72, 100, 128, 500, 512, 513, 1024, 4096, 70000, 1 << 22]
    seqs = [1, 2, 3, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 100, 128, 512, 4096]
    size = {(t, n): L.draft_layer_workspace_bytes(t, n, hq, hkv, d) for t in rows for n in seqs}
    for at, here in (((i, j), size[t, n]) for i, t in enumerate(rows) for j, n in enumerate(seqs)):
        i, j = at
        assert i == 0 or here >= size[rows[i - 1], seqs[j]], at
        assert j == 0 or here >= size[rows[i], seqs[j - 1]], at


@pytest.mark.parametrize("hq,hkv,d", [(40, 8, 128), (7, 7, 256), (16, 1, 64)])
@pytest.mark.parametrize("most_rows,most_seqs", [(512, 64), (4096, 1), (64, 64), (20, 4)])
def test_attend_takes_the_largest_batchs_workspace(lib, hq, hkv, d, most_rows, most_seqs):
    """No smaller call asks for more than the size for the largest batch (what a
    call asks for is in its refusal of a workspace of 16 bytes)."""
    given = L.draft_layer_workspace_bytes(most_rows, most_seqs, hq, hkv, d)
    for t in (1, 2, 5, 17, 64, 65, 500, 512, 4096):
        for n in (1, 2, 3, 8, 63, 64):
            if t <= most_rows and n <= most_seqs:
                _refused(lib, lib.draft_layer_attend, ATTEND,
                         dict(T=t, n_seq=n, hq=hq, hkv=hkv, D=d, ldq=hq * d, bytes=16), B.DH_EINVAL, b"attend")
                need = int(re.search(rb"below the (\d+) needed", lib.draft_head_last_error()).group(1))
                assert 16 < need <= given, (t, n)


def test_kernel_attributes_are_set_on_every_device(tmp_path):
    """A kernel's LDS limit is set once a device, from any number of threads, and
    again after a failure (the helper alone, with counters in the runtime's place)."""
    csrc = os.path.join(os.path.dirname(B.__file__), "csrc")
    src = tmp_path / "once.cpp"
    src.write_text(r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "common.h"
int main() {
  dh::OncePerDevice once;
  std::atomic<int> calls[80] = {};
  auto on = [&](int device, int result) { return once.run(device, 0, [&] { ++calls[device]; return result; }); };
  if (on(0, 7) != 7 || on(0, 7) != 7 || calls[0] != 2) return 1;     // failed: tried again
  for (int i = 0; i < 3; ++i)
    for (int d : {0, 1, 63}) if (on(d, 0) != 0) return 2;
  if (calls[0] != 3 || calls[1] != 1 || calls[63] != 1) return 3;    // once each
  for (int i = 0; i < 3; ++i) on(64, 0);
  if (calls[64] != 3) return 4;                                      // more devices than it remembers
  std::vector<std::thread> pool;
  for (int t = 0; t < 8; ++t) pool.emplace_back([&] { for (int i = 0; i < 1000; ++i) on(i % 32 + 2, 0); });
  for (auto& t : pool) t.join();
  for (int d = 2; d < 34; ++d) if (calls[d] < 1 || calls[d] > 8) return 5;
  return 0;
}
""")
    exe = tmp_path / "once"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
    for name in ("layer_attend.hip", "layer_cache.hip"):
        with open(os.path.join(csrc, name)) as f:
            assert "hipFuncSetAttribute" not in f.read()     # through the helper alone
