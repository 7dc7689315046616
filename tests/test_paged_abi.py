"""Refusals of the paged serving calls: every one is checked on the host,
before any CUDA call (the pointers here are numbers that no GPU has seen)."""
import ctypes

import pytest

A = 0x10000            # an aligned stand-in for a device pointer


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


def assign(kv, **over):
    a = dict(device=0, R=4, held=A, lens=A, free=A, n_free=8, head=A,
             table=A, max_blocks=4, block_size=16, slots=A, slot_capacity=9,
             cu=A, held_out=A, head_out=A, workspace=A,
             workspace_bytes=1 << 20, flags=None, stream=None)
    a.update(over)
    return kv.lib().kvtc_paged_assign(*a.values())


def append(kv, **over):
    a = dict(device=0, n=2, src=[A, A], ld=128, N=3, slots=A, D=128,
             block_size=16, cache=[A, A], num_blocks=4, flags=None,
             stream=None)
    a.update(over)
    for key in ("src", "cache"):
        if a[key] is not None:
            a[key] = (ctypes.c_void_p * max(1, len(a[key])))(*a[key])
    return kv.lib().kvtc_paged_append(*a.values())


def attend(kv, **over):
    a = dict(device=0, R=2, heads=8, kv_heads=2, head_dim=128, dtype=0, q=A,
             q_ld=1024, k=A, v=A, num_blocks=4, block_size=16, table=A,
             max_blocks=2, lens=A, sink=0, window=0, scale=0.1, out=A,
             out_ld=1024, lse=A, workspace=A, workspace_bytes=1 << 30,
             flags=None, stream=None)
    a.update(over)
    return kv.lib().kvtc_paged_attend(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(device=-1), "EINVAL"), (dict(R=-1), "EINVAL"),
    (dict(R=4097), "EINVAL"), (dict(held=None), "EINVAL"),
    (dict(lens=None), "EINVAL"), (dict(free=None), "EINVAL"),
    (dict(n_free=-1), "EINVAL"), (dict(head=None), "EINVAL"),
    (dict(table=None), "EINVAL"), (dict(max_blocks=0), "EINVAL"),
    (dict(slots=None), "EINVAL"), (dict(slot_capacity=-1), "EINVAL"),
    (dict(cu=None), "EINVAL"), (dict(held_out=None), "EINVAL"),
    (dict(head_out=None), "EINVAL"), (dict(workspace=None), "EINVAL"),
    (dict(block_size=32), "ENOTSUP"), (dict(workspace_bytes=16), "ESIZE"),
    (dict(held=A + 2), "EALIGN"), (dict(lens=A + 2), "EALIGN"),
    (dict(free=A + 2), "EALIGN"), (dict(head=A + 4), "EALIGN"),
    (dict(table=A + 2), "EALIGN"), (dict(slots=A + 4), "EALIGN"),
    (dict(cu=A + 4), "EALIGN"), (dict(held_out=A + 2), "EALIGN"),
    (dict(head_out=A + 4), "EALIGN"), (dict(workspace=A + 8), "EALIGN"),
    (dict(flags=A + 2), "EALIGN")])
def test_assign_refusals(kv, over, code):
    assert assign(kv, **over) == getattr(kv, "KVTC_" + code)


@pytest.mark.parametrize("over,code", [
    (dict(device=-1), "EINVAL"), (dict(n=-1), "EINVAL"),
    (dict(src=None), "EINVAL"), (dict(cache=None), "EINVAL"),
    (dict(src=[A, None]), "EINVAL"), (dict(cache=[None, A]), "EINVAL"),
    (dict(N=-1), "EINVAL"), (dict(N=1 << 31), "EINVAL"),
    (dict(slots=None), "EINVAL"), (dict(D=0), "EINVAL"),
    (dict(num_blocks=0), "EINVAL"), (dict(num_blocks=1 << 31), "EINVAL"),
    (dict(D=12, ld=16), "ENOTSUP"), (dict(D=8200, ld=8200), "ENOTSUP"),
    (dict(block_size=8), "ENOTSUP"), (dict(ld=120), "ESIZE"),
    (dict(ld=132), "EALIGN"), (dict(slots=A + 4), "EALIGN"),
    (dict(src=[A, A + 8]), "EALIGN"), (dict(cache=[A + 8, A]), "EALIGN"),
    (dict(flags=A + 1), "EALIGN")])
def test_append_refusals(kv, over, code):
    assert append(kv, **over) == getattr(kv, "KVTC_" + code)


@pytest.mark.parametrize("over,code", [
    (dict(device=-1), "EINVAL"), (dict(R=-1), "EINVAL"),
    (dict(R=4097), "EINVAL"), (dict(heads=0), "EINVAL"),
    (dict(kv_heads=0), "EINVAL"), (dict(heads=9), "EINVAL"),
    (dict(head_dim=0), "EINVAL"), (dict(dtype=2), "EINVAL"),
    (dict(q=None), "EINVAL"), (dict(k=None), "EINVAL"),
    (dict(v=None), "EINVAL"), (dict(table=None), "EINVAL"),
    (dict(lens=None), "EINVAL"), (dict(out=None), "EINVAL"),
    (dict(workspace=None), "EINVAL"), (dict(num_blocks=0), "EINVAL"),
    (dict(num_blocks=1 << 31), "EINVAL"), (dict(max_blocks=0), "EINVAL"),
    (dict(sink=-1), "EINVAL"), (dict(window=-1), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"),
    (dict(scale=float("inf")), "EINVAL"),
    (dict(block_size=32), "ENOTSUP"), (dict(head_dim=96), "ENOTSUP"),
    (dict(max_blocks=(1 << 27) - 1), "ENOTSUP"),
    (dict(heads=80, kv_heads=80, q_ld=10240, out_ld=10240), "ENOTSUP"),
    (dict(heads=129, kv_heads=1, q_ld=16512, out_ld=16512), "ENOTSUP")])
def test_attend_refusals(kv, over, code):
    assert attend(kv, **over) == getattr(kv, "KVTC_" + code)


@pytest.mark.parametrize("over,code", [
    (dict(q_ld=1016), "ESIZE"), (dict(out_ld=1016), "ESIZE"),
    (dict(workspace_bytes=8), "ESIZE"), (dict(q_ld=1028), "EALIGN"),
    (dict(out_ld=1028), "EALIGN"), (dict(q=A + 8), "EALIGN"),
    (dict(k=A + 8), "EALIGN"), (dict(v=A + 8), "EALIGN"),
    (dict(out=A + 8), "EALIGN"), (dict(workspace=A + 8), "EALIGN"),
    (dict(table=A + 2), "EALIGN"), (dict(lens=A + 2), "EALIGN"),
    (dict(lse=A + 2), "EALIGN"), (dict(flags=A + 2), "EALIGN")])
def test_attend_sizes_and_alignment(kv, over, code):
    assert attend(kv, **over) == getattr(kv, "KVTC_" + code)


@pytest.mark.parametrize("scale,fine", [
    (3.4e38, False), (-3.4e38, False), (1.8e38, False),
    (float("-inf"), False), (2.0 ** 127, True), (-2.0 ** 127, True),
    (0.0, True), (1e-45, True)])
def test_attend_scale(kv, scale, fine):
    """scale log2(e) has to be finite in fp32: an infinite one makes NaN of
    a score that is zero."""
    assert attend(kv, R=0, scale=scale) == (kv.KVTC_OK if fine
                                            else kv.KVTC_EINVAL)


def test_workspace_queries(kv):
    L = kv.lib()
    assert L.kvtc_paged_assign_workspace_bytes(-1) == kv.KVTC_EINVAL
    assert L.kvtc_paged_assign_workspace_bytes(4097) == kv.KVTC_EINVAL
    assert L.kvtc_paged_assign_workspace_bytes(4096) > 0
    for args, code in (((-1, 1, 1, 1, 64), kv.KVTC_EINVAL),
                       ((0, 4097, 1, 1, 64), kv.KVTC_EINVAL),
                       ((0, 1, 3, 2, 64), kv.KVTC_EINVAL),
                       ((0, 1, 2, 2, 72), kv.KVTC_ENOTSUP)):
        assert L.kvtc_paged_attend_workspace_bytes(*args) == code


def test_empty_calls_are_accepted_before_any_cuda_call(kv):
    assert append(kv, N=0, slots=None, src=[None, None]) == kv.KVTC_OK
    assert append(kv, n=0, src=[], cache=[]) == kv.KVTC_OK
    assert attend(kv, R=0, q=None, table=None, lens=None, out=None) == \
        kv.KVTC_OK


def test_binding_raises(kv):
    with pytest.raises(kv.KvtcError) as e:
        kv.kvtc_paged_append([A], 4, 1, A, 8, 16, [A], 1, stream=0)
    assert e.value.code == kv.KVTC_ESIZE
    with pytest.raises(ValueError):
        kv.kvtc_paged_append([A], 8, 1, A, 8, 16, [], 1, stream=0)
    with pytest.raises(kv.KvtcError) as e:
        kv.kvtc_paged_attend(1, 2, 3, 64, 0, A, 128, A, A, 1, 16, A, 1, A, 0,
                             0, 1.0, A, 128, None, A, 1 << 30, stream=0)
    assert e.value.code == kv.KVTC_EINVAL


class OnDevice:
    """Stands in for a tensor."""

    def __init__(self, device):
        self.device = device

    def data_ptr(self):
        return A

    def get_device(self):
        return self.device


@pytest.mark.parametrize("where,given,used", [
    (1, None, 1), (0, None, 0), (3, 2, 2), (None, None, 0), (None, 5, 5),
    (-1, None, 0)])
def test_calls_run_on_their_tensors_device(kv, monkeypatch, where, given,
                                           used):
    """By default, on the device of the table or the pools, whatever device
    is current; a launch on device 0 could not read them."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args[0])) or 0
    monkeypatch.setattr(kv, "_lib_handle", Lib())
    x = A if where is None else OnDevice(where)
    more = dict(stream=0, **({} if given is None else {"device": given}))
    kv.kvtc_paged_assign(1, x, x, x, 1, x, x, 1, 16, x, 1, x, x, x, x, 256,
                         **more)
    kv.kvtc_paged_append([x], 8, 1, x, 8, 16, [x], 1, **more)
    kv.kvtc_paged_attend(1, 1, 1, 64, 0, x, 64, x, x, 1, 16, x, 1, x, 0, 0,
                         1.0, x, 64, None, x, 1 << 20, **more)
    kv.kvtc_paged_append([], 8, 0, None, 8, 16, [], 1, **more)
    assert seen == [("kvtc_paged_assign", used), ("kvtc_paged_append", used),
                    ("kvtc_paged_attend", used),
                    ("kvtc_paged_append", given or 0)]
