"""Edges of the rotary and grouped-query calls that need no GPU: sizes,
refusals, and the state of the binding."""
import ctypes
import os
import random
import re
import subprocess
import sys
import sysconfig
import threading
import warnings

import pytest

import paged_kv_cache_269_gb300 as pa
from paged_kv_cache_269_gb300 import grouped
from paged_kv_cache_269_gb300.grouped import AttnOpts


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_counters_hold_a_word_for_every_unit(D):
    """Each (sequence, K/V head, chunk of query heads) has a ticket of its own."""
    for S in list(range(0, 301)) + [4095, 4096]:
        for H, group in ((1, 1), (1, 9), (3, 8), (7, 4), (8, 17), (1, 71)):
            per = 16 if group > 8 and D != 256 else 8
            units = S * H * -(-group // per)
            n = pa.decode_grouped_counters_bytes(S, H * group, H, D, 16)
            assert n % 256 == 0 and n >= max(4 * units, 256)
            assert n < 4 * units + 512


def _ahead(items, slots, bufs, descending, held_tile, held):
    """How far past key tile `held` the K copies of the grouped prefill get while the
    softmax of query tile `held_tile` stands there and every other role goes on as
    far as its waits allow.  items: (key tiles, those tile 0 needs, those tile 1
    needs or -1)."""
    needs = []
    for n, n0, n1 in items:
        for j in range(n):
            at = n - 1 - j if descending else j
            needs.append((at < n0, at < n1))
    total = len(needs)
    own = [[i for i in range(total) if needs[i][t]] for t in (0, 1)]
    if held not in own[held_tile]:
        return 0
    k = v = 0                                     # tiles of K and V loaded
    s, pv = [0, 0], [0, 0]                        # tiles passed by the product threads
    scores, weights, products = [0, 0], [0, 0], [0, 0]
    while True:
        before = (k, v, *s, *pv, *weights)
        while k < total and (k < slots or min(s) > k - slots):
            k += 1
        while v < total and (v < slots or min(pv) > v - slots):
            v += 1
        for t in (0, 1):
            while s[t] < k and not (needs[s[t]][t] and scores[t] - products[t] >= bufs):
                scores[t] += needs[s[t]][t]
                s[t] += 1
            while weights[t] < scores[t] and not (t == held_tile and own[t][weights[t]] == held):
                weights[t] += 1
            while pv[t] < v and not (needs[pv[t]][t] and products[t] >= weights[t]):
                products[t] += needs[pv[t]][t]
                pv[t] += 1
        if before == (k, v, *s, *pv, *weights):
            return k - 1 - held


def test_prefill_mask_ring_outlasts_its_slowest_reader():
    """A key tile's entry is rewritten one ring later, without a wait: no order of
    the roles may bring the copies that far ahead of a softmax yet to read it."""
    path = os.path.join(os.path.dirname(pa.__file__), "csrc", "pa_prefill_grouped.cu")
    src = open(path).read()
    ring = int(re.search(r"kMaskRing = (\d+);", src).group(1))
    slots = re.search(r"kSlots = D == 64 \? (\d+) : (\d+);", src).groups()
    bufs = re.search(r"kBufs = D == 64 \? (\d+) : (\d+);", src).groups()
    rng = random.Random(1)
    for ns, nb in zip(map(int, slots), map(int, bufs)):
        most = 0
        for _ in range(6000):
            items = []
            for _ in range(rng.randint(2, 8)):
                n = rng.choice([1, 1, 2, 2, 3, 4, 8, 16, 17])
                items.append((n, n, -1) if rng.random() < 0.5 else (n, max(0, n - rng.randint(0, 3)), n))
            tiles = sum(i[0] for i in items)
            most = max(most, _ahead(items, ns, nb, rng.random() < 0.5, rng.randint(0, 1), rng.randrange(tiles)))
        assert 0 < most <= 2 * ns + 2 * nb - 2    # the bound that the kernel asserts
        assert most < ring


FAKE = ctypes.c_void_p(0x100000)     # never dereferenced: the checks fail first


def test_scales_and_caps_that_fp32_cannot_hold_are_refused():
    lib = pa.lib()

    def refused(scale, cap):
        d, o = pa.Dims(2, 4, 128, 16, 32, 0), AttnOpts(cap, 0, None, None)
        # no counters: a call that the numbers do not stop is stopped there (-5)
        rc = {lib.pa_decode_grouped(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, scale, 8, ctypes.byref(d), 8, ctypes.byref(o),
                                    FAKE, 1 << 30, None, 0, None),
              lib.pa_prefill_grouped(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 4, scale, 8, ctypes.byref(d), 8,
                                     ctypes.byref(o), FAKE, 1 << 30, None, 0, None)}
        assert rc in ({-2}, {-5})
        return rc == {-2}

    assert refused(3e38, 0.0) and refused(-3e38, 0.0) and refused(float("inf"), 0.0)
    assert refused(0.1, 1e-39) and refused(0.1, 1e-31) and refused(0.1, 3e38)
    assert refused(1e25, 1e-25) and refused(1e-20, 1e15)
    assert not refused(1e30, 0.0) and not refused(0.0, 50.0) and not refused(-0.1, 50.0)
    assert not refused(0.1, 1e-25) and not refused(0.1, 1e25) and not refused(1e-38, 0.0)


def test_numbers_past_32_bits_are_not_cut():
    """A bound that 32 bits do not hold bounds nothing; it does not become its low
    32 bits.  A cap that fp32 would take for 0, which says none, is refused."""
    top = 2 ** 31 - 1
    for n in (0, 1, 1024, top):
        assert grouped._bound(n, "window") == n
    for n in (top + 1, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 80):
        assert grouped._bound(n, "window") == top
    for n in (-1, -2 ** 31 - 7, -2 ** 32):
        assert grouped._bound(n, "window") == -1          # the library refuses it
    assert grouped._bound(7.0, "window") == 7
    with pytest.raises(ValueError):
        grouped._bound(0.5, "window")
    assert grouped._cap(None) == 0.0 and grouped._cap(0) == 0.0 and grouped._cap(30) == 30.0
    assert grouped._cap(-2.0) == -2.0                      # the library refuses it
    with pytest.raises(ValueError):
        grouped._cap(1e-50)


@pytest.fixture
def fresh_binding(monkeypatch):
    """The binding as a process finds it before its first grouped call, on a machine
    that says it has CUDA."""
    torch = pytest.importorskip("torch")
    for name in ("torch", "Tensor", "_I32", "_F32", "_U8", "_raw_stream", "_package", "_marshal", "_get_device",
                 "_capturing"):
        monkeypatch.setattr(grouped, name, None)
    monkeypatch.setattr(grouped, "_buffers", {})
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    if not hasattr(torch._C, "_cuda_getCurrentRawStream"):
        pytest.skip("a torch without CUDA")
    return monkeypatch


def test_a_marshalling_module_that_does_not_build_is_told_once(fresh_binding):
    calls = []

    def broken():
        calls.append(1)
        raise RuntimeError("no compiler")

    fresh_binding.setattr(pa._build, "build_marshal", broken)
    with pytest.warns(RuntimeWarning, match="no compiler"):
        assert grouped._pa() is pa
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert grouped._pa() is pa
    assert calls == [1] and grouped._marshal is None and grouped._raw_stream is not None


def test_a_second_thread_waits_for_the_first_call(fresh_binding):
    building, go = threading.Event(), threading.Event()

    def slow():
        building.set()
        assert go.wait(30)
        return "path"

    module = object()
    fresh_binding.setattr(pa._build, "build_marshal", slow)
    fresh_binding.setattr(grouped, "_load_marshal", lambda path: module)
    found = []

    def call():
        package = grouped._pa()
        found.append((package, grouped._raw_stream is not None, grouped._marshal))

    threads = [threading.Thread(target=call) for _ in range(4)]
    threads[0].start()
    assert building.wait(30)
    for t in threads[1:]:
        t.start()
    threads[1].join(0.2)
    assert found == []
    go.set()
    for t in threads:
        t.join(30)
    assert found == [(pa, True, module)] * 4


def test_resetting_workspaces_builds_nothing(fresh_binding):
    def never():
        raise AssertionError("built")

    fresh_binding.setattr(pa._build, "build_marshal", never)
    pa.reset_workspaces()
    assert grouped._package is None


def test_the_marshalling_module_belongs_to_one_torch_and_python(monkeypatch):
    torch = pytest.importorskip("torch")
    path = pa._build.marshal_path()
    assert os.path.dirname(path) == pa._build.LIB_DIR and path.endswith(".so")
    monkeypatch.setattr(torch, "__version__", "0.0+other")
    other = pa._build.marshal_path()
    assert other != path
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-00")
    assert pa._build.marshal_path() not in (path, other)


_WITHOUT_STORAGE = """
import ctypes, sys
import torch
import paged_kv_cache_269_gb300 as pa
from paged_kv_cache_269_gb300 import grouped

class Held(torch.Tensor):            # says that it is a CUDA tensor, holds nothing
    @staticmethod
    def __new__(cls, dtype, *size):
        return torch.Tensor._make_wrapper_subclass(cls, size, dtype=dtype, device="cuda:0")
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)

module, lib = grouped._load_marshal(pa._build.build_marshal()), pa.lib()
def at(name):
    return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
half, whole = torch.float16, torch.int32
shapes = [(half, 2, 4, 128), (half, 2, 4, 128), (half, 2, 2, 128), (half, 2, 2, 128), (half, 8, 2, 16, 128),
          (half, 8, 2, 16, 128), (whole, 2, 4), (whole, 2), (whole, 3), (whole, 4096), (torch.uint8, 1 << 24),
          (torch.float32, 9, 128)]
found = []
def calls(out, q, k, v, kc, vc, tables, lens, starts, counters, workspace, table):
    common = (out, q, kc, vc, tables, lens, 0.1, 0.0, None, 0, None, counters, workspace, 0, 0)
    found.append(module.decode(*common, at("pa_decode_grouped"), at("pa_decode_grouped_workspace_bytes"),
                               at("pa_decode_grouped_counters_bytes")))
    found.append(module.prefill(*common, starts, 1, at("pa_prefill_grouped"), at("pa_prefill_grouped_workspace_bytes"),
                                at("pa_prefill_grouped_counters_bytes")))
    found.append(module.rope(out, q, k, v, kc, vc, lens, table, lens, False, 0, 0, at("pa_rope_and_cache")))
    raise StopIteration
try:
    torch.vmap(calls)(*[Held(s[0], 1, *s[1:]) for s in shapes])
except StopIteration:
    pass
assert found == [None] * 3, found
"""


def test_marshalled_calls_hand_back_tensors_without_storage():
    """A batched tensor of vmap has no address to give, and asking for one throws:
    the call goes to the Python checks, the interpreter stays alive."""
    pytest.importorskip("torch")
    r = subprocess.run([sys.executable, "-c", _WITHOUT_STORAGE], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(pa.__file__)))
    assert r.returncode == 0, r.stderr[-2000:]
