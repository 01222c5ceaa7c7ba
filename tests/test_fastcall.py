"""The extension that passes plain numbers to the C entry points: every argument
arrives as it was given, in its place and type (a recording function stands in
for the library's), and what does not fit is refused."""
import ctypes

import pytest

from paged_kv_cache_480_b200 import binding

NAMES = ("rotary_embedding", "rotary_reshape_and_cache", "rotary_reshape_and_cache_fp8row", "reshape_and_cache_fp8row",
         "gather_cache", "gather_cache_fp8kv", "gather_cache_fp8row", "paged_attention_decode_fp8row",
         "paged_attention_prefill_fp8row", "paged_attention_prefill_fp8kv", "paged_attention_workspace_size")


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


class Recorder:
    """Stands in for one entry point while it is alive."""

    def __init__(self, lib, name, result=0):
        fn = getattr(lib, name)
        self.types, self.name, self.got = fn.argtypes, name, []
        self.callback = ctypes.CFUNCTYPE(fn.restype, *fn.argtypes)(lambda *a: self.got.append(a) or result)
        self.address = ctypes.cast(fn, ctypes.c_void_p).value

    def __enter__(self):
        binding._fast.bind(self.name, ctypes.cast(self.callback, ctypes.c_void_p).value)
        return self

    def __exit__(self, *exc):
        binding._fast.bind(self.name, self.address)

    def values(self):
        """A different value for each argument, the widest that its type takes among them."""
        out = []
        for i, t in enumerate(self.types):
            out.append({ctypes.c_void_p: (1 << 47) + 16 * i, ctypes.c_int: (1 << 31) - 1 - i,
                        ctypes.c_int64: -(1 << 62) + i, ctypes.c_size_t: (1 << 40) + i, ctypes.c_float: 0.5 + i}[t])
        return out


@pytest.mark.parametrize("name", NAMES)
def test_arguments_arrive(lib, name):
    with Recorder(lib, name, 7) as r:
        v = r.values()
        # dtypes are passed as the three codes of the enum
        if name == "paged_attention_workspace_size":
            v[6] = 2
        else:
            at = len(v) - (5 if "decode" in name else 2)
            v[at] = 2
        assert getattr(binding._fast, name)(*v) == 7
        assert list(r.got[0]) == v
        null = [None if t is ctypes.c_void_p else x for t, x in zip(r.types, v)]
        getattr(binding._fast, name)(*null)
        assert list(r.got[1]) == null


@pytest.mark.parametrize("name", NAMES)
def test_refusals(lib, name):
    with Recorder(lib, name) as r:
        v = r.values()
        fn = getattr(binding._fast, name)
        with pytest.raises(TypeError):
            fn(*v[:-1])
        with pytest.raises(TypeError):
            fn(*v, 0)
        for i, t in enumerate(r.types):
            bad = list(v)
            bad[i] = "1"
            with pytest.raises(TypeError):
                fn(*bad)
            if t is ctypes.c_int:
                bad[i] = 1 << 31
                with pytest.raises(OverflowError):
                    fn(*bad)
        assert r.got == []


def test_bind_refuses_other_names(lib):
    with pytest.raises(ValueError):
        binding._fast.bind("copy_blocks", 0)


def test_same_status_as_ctypes(lib):
    """A refused size and a null pointer give the status that ctypes gives."""
    for name in NAMES[:-1]:
        zero = [None if t is ctypes.c_void_p else 0 for t in getattr(lib, name).argtypes]
        assert getattr(binding._fast, name)(*zero) == getattr(lib, name)(*zero)
    assert binding._fast.paged_attention_workspace_size(8, 8, 8, 64, 16, 512, 1, 0) == \
        lib.paged_attention_workspace_size(8, 8, 8, 64, 16, 512, 1, 0)
