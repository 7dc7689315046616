"""Refusals of the calls around chunks of new tokens: every one is checked on
the host, before any CUDA call (the pointers here are numbers that no GPU has
seen); rotary frequencies against their formulas."""
import ctypes
import math

import pytest

A = 0x10000            # an aligned stand-in for a device pointer
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def kv():
    from kv_cache_transform_gb300 import _build
    _build.build()
    import kv_cache_transform_gb300 as kv
    return kv


def rotate(kv, **over):
    a = dict(device=0, N=3, heads=8, kv_heads=2, head_dim=128, dtype=0, q=A,
             k=A, v=A, ld=1536, positions=A, inv_freq=A, rotary_dim=128,
             interleaved=0, scale=1.0, q_norm=A, k_norm=A, eps=1e-6, q_out=A,
             q_out_ld=1024, slots=A, block_size=16, k_cache=A, v_cache=A,
             num_blocks=4, flags=None, stream=None)
    a.update(over)
    return kv.lib().kvtc_paged_rotate(*a.values())


def chunks(kv, **over):
    a = dict(device=0, R=2, N=9, heads=8, kv_heads=2, head_dim=128, dtype=0,
             q=A, q_ld=1024, k=A, v=A, num_blocks=4, block_size=16, table=A,
             max_blocks=2, cu=A, lens=A, sink=0, window=0, scale=0.1, out=A,
             out_ld=1024, lse=A, workspace=A, workspace_bytes=1 << 40,
             flags=None, stream=None)
    a.update(over)
    return kv.lib().kvtc_paged_attend_chunks(*a.values())


def weigh(kv, **over):
    a = dict(device=0, R=2, N=9, heads=8, kv_heads=2, head_dim=128, dtype=0,
             q=A, q_ld=1024, k=A, num_blocks=4, block_size=16, table=A,
             max_blocks=2, cu=A, lens=A, sink=0, window=0, scale=0.1, lse=A,
             decay=1.0, acc=A, acc_out=A, acc_ld=32, workspace=A,
             workspace_bytes=1 << 40, flags=None, stream=None)
    a.update(over)
    return kv.lib().kvtc_paged_weigh(*a.values())


def evict(kv, **over):
    a = dict(device=0, R=2, acc=A, acc_ld=32, lens=A, keep=20, sink=4,
             window=8, table=A, out_table=A, max_blocks=2, block_size=16,
             n=2, cache=[A, A], D=128, num_blocks=4, kept=A, acc_out=A,
             lens_out=A, workspace=A, workspace_bytes=1 << 40, flags=None,
             stream=None)
    a.update(over)
    if a["cache"] is not None:
        a["cache"] = (ctypes.c_void_p * max(1, len(a["cache"])))(*a["cache"])
    return kv.lib().kvtc_paged_evict(*a.values())


@pytest.mark.parametrize("code,overs", [
    ("EINVAL", [dict(device=-1), dict(N=-1), dict(N=1 << 31), dict(heads=0),
                dict(kv_heads=0), dict(head_dim=0), dict(dtype=2),
                dict(q=None), dict(k=None), dict(v=None), dict(v_cache=None),
                dict(positions=None), dict(inv_freq=None),
                dict(rotary_dim=-8), dict(rotary_dim=136), dict(scale=NAN),
                dict(scale=INF), dict(eps=-1.0), dict(eps=NAN),
                dict(eps=INF), dict(q_out=None), dict(slots=None),
                dict(k_cache=None), dict(num_blocks=0),
                dict(num_blocks=1 << 31)]),
    ("ENOTSUP", [dict(block_size=8), dict(rotary_dim=4),
                 dict(head_dim=96, rotary_dim=96), dict(kv_heads=65, ld=65 * 128),
                 dict(heads=1025, ld=1025 * 128, q_out_ld=1025 * 128)]),
    ("ESIZE", [dict(ld=1016), dict(q_out_ld=1016),
               dict(kv_heads=16, heads=4, ld=1024)]),
    ("EALIGN", [dict(ld=1540), dict(q_out_ld=1028), dict(q=A + 8),
                dict(k=A + 8), dict(v=A + 8), dict(q_out=A + 8),
                dict(k_cache=A + 8), dict(v_cache=A + 8),
                dict(q_norm=A + 2), dict(k_norm=A + 2),
                dict(positions=A + 2), dict(inv_freq=A + 4),
                dict(slots=A + 4), dict(flags=A + 2)])])
def test_rotate_refusals(kv, code, overs):
    for over in overs:
        assert rotate(kv, **over) == getattr(kv, "KVTC_" + code), over


SHAPES = [
    ("EINVAL", [dict(device=-1), dict(R=-1), dict(R=4097), dict(N=-1),
                dict(N=1 << 31), dict(heads=0), dict(kv_heads=0),
                dict(heads=9), dict(head_dim=0), dict(dtype=2),
                dict(q=None), dict(k=None), dict(table=None), dict(cu=None),
                dict(lens=None), dict(workspace=None), dict(num_blocks=0),
                dict(num_blocks=1 << 31), dict(max_blocks=0), dict(sink=-1),
                dict(window=-1), dict(scale=NAN), dict(scale=-INF),
                dict(scale=1.8e38)]),
    ("ENOTSUP", [dict(block_size=32), dict(head_dim=96),
                 dict(max_blocks=(1 << 27) - 1, acc_ld=1 << 31),
                 dict(heads=80, kv_heads=80, q_ld=10240, out_ld=10240),
                 dict(heads=129, kv_heads=1, q_ld=16512, out_ld=16512)]),
    ("ESIZE", [dict(q_ld=1016), dict(workspace_bytes=8)]),
    ("EALIGN", [dict(q_ld=1028), dict(q=A + 8), dict(k=A + 8),
                dict(workspace=A + 8), dict(table=A + 2), dict(cu=A + 4),
                dict(lens=A + 2), dict(lse=A + 2), dict(flags=A + 2)])]


@pytest.mark.parametrize("call", [chunks, weigh])
@pytest.mark.parametrize("code,overs", SHAPES)
def test_shape_refusals(kv, call, code, overs):
    for over in overs:
        other = ("acc_ld",) if call is chunks else ("out_ld",)
        over = {k: x for k, x in over.items() if k not in other}
        assert call(kv, **over) == getattr(kv, "KVTC_" + code), over


@pytest.mark.parametrize("code,overs", [
    ("EINVAL", [dict(v=None), dict(out=None)]),
    ("ESIZE", [dict(out_ld=1016)]),
    ("EALIGN", [dict(v=A + 8), dict(out=A + 8), dict(out_ld=1028)])])
def test_chunk_refusals(kv, code, overs):
    for over in overs:
        assert chunks(kv, **over) == getattr(kv, "KVTC_" + code), over


@pytest.mark.parametrize("code,overs", [
    ("EINVAL", [dict(lse=None), dict(decay=NAN), dict(decay=INF),
                dict(acc=None), dict(acc_out=None)]),
    ("ESIZE", [dict(acc_ld=28)]),
    ("EALIGN", [dict(acc_ld=34), dict(acc=A + 8), dict(acc_out=A + 8)])])
def test_weigh_refusals(kv, code, overs):
    for over in overs:
        assert weigh(kv, **over) == getattr(kv, "KVTC_" + code), over


@pytest.mark.parametrize("code,overs", [
    ("EINVAL", [dict(device=-1), dict(R=-1), dict(R=4097), dict(acc=None),
                dict(lens=None), dict(keep=-1), dict(keep=11), dict(sink=-1),
                dict(window=-1), dict(table=None), dict(out_table=None),
                dict(max_blocks=0), dict(n=-1), dict(cache=None),
                dict(cache=[A, None]), dict(D=0), dict(num_blocks=0),
                dict(num_blocks=1 << 31), dict(kept=None),
                dict(acc_out=None), dict(lens_out=None),
                dict(workspace=None),
                dict(sink=2 ** 31 - 1, window=2 ** 31 - 1)]),
    ("ENOTSUP", [dict(block_size=8), dict(D=12), dict(D=8200),
                 dict(max_blocks=(1 << 27) - 1, acc_ld=1 << 31)]),
    ("ESIZE", [dict(acc_ld=28), dict(workspace_bytes=8)]),
    ("EALIGN", [dict(acc_ld=34), dict(acc=A + 4), dict(acc_out=A + 4),
                dict(lens=A + 2), dict(table=A + 2), dict(out_table=A + 2),
                dict(kept=A + 2), dict(lens_out=A + 2),
                dict(cache=[A + 8, A]), dict(workspace=A + 8),
                dict(flags=A + 2)])])
def test_evict_refusals(kv, code, overs):
    for over in overs:
        assert evict(kv, **over) == getattr(kv, "KVTC_" + code), over


def test_empty_calls(kv):
    assert rotate(kv, N=0, q=None, k=None, v=None, slots=None, q_out=None,
                  positions=None) == kv.KVTC_OK
    assert chunks(kv, N=0, q=None, out=None) == kv.KVTC_OK
    assert chunks(kv, R=0, N=0, q=None, out=None, table=None, cu=None,
                  lens=None) == kv.KVTC_OK
    assert weigh(kv, R=0, N=0, q=None, lse=None, table=None, cu=None,
                 lens=None, acc_out=None) == kv.KVTC_OK
    assert evict(kv, R=0, acc=None, lens=None, table=None, out_table=None,
                 kept=None, acc_out=None, lens_out=None) == kv.KVTC_OK


def test_workspace_queries(kv):
    with pytest.raises(kv.KvtcError):
        kv.kvtc_paged_attend_chunks_workspace_bytes(4097, 9, 8, 2, 128)
    with pytest.raises(kv.KvtcError):
        kv.kvtc_paged_weigh_workspace_bytes(2, 9, 8, 2, 96)
    with pytest.raises(kv.KvtcError):
        kv.kvtc_paged_evict_workspace_bytes(2, 0)
    assert kv.kvtc_paged_evict_workspace_bytes(0, 1) > 0
    assert kv.kvtc_paged_attend_chunks_workspace_bytes(0, 0, 8, 2, 128) > 0


def test_frequencies(kv):
    f = kv.kvtc_rotary_frequencies(8, 10000.0)
    assert f == pytest.approx([1, 0.1, 0.01, 0.001], rel=1e-14)
    g = kv.kvtc_rotary_frequencies(8, 10000.0, kv.KVTC_ROTARY_LINEAR, 4.0)
    assert g == pytest.approx([x / 4 for x in f], rel=1e-14)
    # the first as it is, the last stretched by the factor
    g = kv.kvtc_rotary_frequencies(8, 10000.0, kv.KVTC_ROTARY_BASE, 4.0)
    assert g[0] == 1 and g[3] == pytest.approx(f[3] / 4, rel=1e-12)
    assert g[1] == pytest.approx((10000 * 4 ** (8 / 6)) ** -0.25, rel=1e-12)
    # 2 pi 100 tokens: 100, 10, 1 and 0.1 turns
    g = kv.kvtc_rotary_frequencies(8, 10000.0, kv.KVTC_ROTARY_BANDS, 8.0,
                                   200 * math.pi, 1.0, 19.0)
    assert g == pytest.approx([1, 0.1 * (0.5 + 0.5 / 8), 0.01 / 8,
                               0.001 / 8], rel=1e-12)


@pytest.mark.parametrize("args", [
    (0, 1e4), (-2, 1e4), (7, 1e4), (8, 0.0), (8, -1.0), (8, INF), (8, NAN),
    (8, 1e4, 4), (8, 1e4, -1), (8, 1e4, 1, 0.0), (8, 1e4, 1, INF),
    (8, 1e4, 2, NAN), (2, 1e4, 2, 2.0), (8, 1e4, 3, 2.0, 0.0, 1.0, 4.0),
    (8, 1e4, 3, 2.0, 100.0, 4.0, 4.0), (8, 1e4, 3, 2.0, 100.0, -1.0, 4.0),
    (8, 1e4, 3, 2.0, 100.0, 1.0, INF), (8, 1e4, 3, 2.0, NAN, 1.0, 4.0)])
def test_frequency_refusals(kv, args):
    with pytest.raises(kv.KvtcError) as e:
        kv.kvtc_rotary_frequencies(*args)
    assert e.value.code == kv.KVTC_EINVAL


def test_frequencies_out_of_range(kv):
    """Frequencies beyond the range of numbers are refused, and nothing is
    written; a stretched base beyond it is no obstacle."""
    for args in ((8, 1e4, kv.KVTC_ROTARY_LINEAR, 1e-310),
                 (8, 1e4, kv.KVTC_ROTARY_BANDS, 1e-310, 100.0, 1.0, 4.0),
                 (256, 5e-324), (4, 1e-300, kv.KVTC_ROTARY_BASE, 1e-200)):
        with pytest.raises(kv.KvtcError) as e:
            kv.kvtc_rotary_frequencies(*args)
        assert e.value.code == kv.KVTC_EINVAL
    out = (ctypes.c_double * 4)(*[77.0] * 4)
    assert kv.lib().kvtc_rotary_frequencies(
        8, 1e4, kv.KVTC_ROTARY_LINEAR, 1e-310, 0.0, 0.0, 0.0,
        out) == kv.KVTC_EINVAL
    assert list(out) == [77.0] * 4
    f = kv.kvtc_rotary_frequencies(4, 1e300, kv.KVTC_ROTARY_BASE, 1e10)
    assert f == pytest.approx([1, 1e-160], rel=1e-12)
