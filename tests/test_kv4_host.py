"""Refusals of the detint_kv4_* entry points and of detint_load_kv that need
no GPU: every argument check comes before the first CUDA call, so made-up
pointers and sizes come back as error codes."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from deterministic_integer_only_gb300 import binding, build
    build.build()
    return binding.lib()


P = 1 << 20     # an aligned address that no refused call touches


def _cache(**kw):
    from deterministic_integer_only_gb300 import binding
    v = dict(n_q=8, n_kv=2, head_dim=64, n_blocks=4, n_seq=2, max_blocks=2, k=P, v=P, k_scale=P, v_scale=P,
             block_table=P, params=P, status=None)
    v.update(kw)
    return binding._Kv4(*[v[n] for n, _ in binding._Kv4._fields_])


def _rope(**kw):
    from deterministic_integer_only_gb300 import binding
    v = dict(cos=P, sin=P, max_pos=64, rot_dim=64, interleaved=0, eps=0, q_gamma=None, k_gamma=None)
    v.update(kw)
    return binding._Rope(*[v[n] for n, _ in binding._Rope._fields_])


def _append(L, c=None, r=None, **kw):
    v = dict(qkv=P, stride=12 * 64, seq=P, pos=P, n=3, q8=P, mq=P, kq=P, kv=None, vv=None)
    v.update(kw)
    c, r = c or _cache(), r or _rope()
    return L.detint_kv4_append(C.addressof(c), C.addressof(r), v["qkv"], v["stride"], v["seq"], v["pos"], v["n"],
                               v["q8"], v["mq"], v["kq"], v["kv"], v["vv"], None)


def _attn(L, which, c=None, **kw):
    v = dict(q8=P, mq=P, kq=P, seq=P, pos=P, n=3, max_len=100, window=0, o=P, stride=8 * 64)
    v.update(kw)
    c = c or _cache()
    a = [C.addressof(c), v["q8"], v["mq"], v["kq"], v["seq"], v["pos"], v["n"], v["max_len"], v["window"], v["o"], v["stride"]]
    return L.detint_kv4_decode(*a, None, 0, None) if which == "decode" else L.detint_kv4_prefill(*a, None)


CACHES = [(1, dict(k=None)), (1, dict(v_scale=None)), (1, dict(params=None)), (1, dict(block_table=None)),
          (2, dict(head_dim=96)), (2, dict(head_dim=0)), (2, dict(n_q=7)), (2, dict(n_kv=0)), (2, dict(n_q=0)),
          (2, dict(n_q=2048)), (2, dict(n_q=130, n_kv=2)), (1, dict(n_blocks=0)), (1, dict(n_seq=-1)), (1, dict(max_blocks=0)),
          (1, dict(k=P + 8)), (1, dict(v_scale=P + 4)), (1, dict(params=P + 4))]


@pytest.mark.parametrize("code,change", CACHES)
def test_bad_caches_are_refused(L, code, change):
    c = _cache(**change)
    n = C.c_longlong(7)
    assert _append(L, c) == code
    assert _attn(L, "decode", c) == code and _attn(L, "prefill", c) == code
    assert L.detint_kv4_workspace(C.addressof(c), 1, 100, C.byref(n)) == code
    assert b"detint_kv4_workspace" in L.detint_last_error()


@pytest.mark.parametrize("code,change", [
    (1, dict(qkv=None)), (1, dict(pos=None)), (1, dict(q8=None)), (1, dict(n=0)), (1, dict(n=-4)), (1, dict(stride=12 * 64 - 4)),
    (1, dict(stride=12 * 64 + 2)), (1, dict(qkv=P + 4)), (1, dict(q8=P + 8)), (1, dict(kv=P + 2)), (1, dict(vv=P + 4))])
def test_bad_append_arguments_are_refused(L, code, change):
    assert _append(L, **change) == code


@pytest.mark.parametrize("code,change", [
    (2, dict(rot_dim=72)), (2, dict(rot_dim=12)), (2, dict(rot_dim=-8)), (1, dict(cos=None)), (1, dict(sin=None)),
    (1, dict(max_pos=0)), (1, dict(interleaved=2)), (1, dict(q_gamma=P)), (1, dict(k_gamma=P)), (1, dict(eps=-1)),
    (1, dict(eps=40000)), (1, dict(cos=P + 4)), (2, dict(max_pos=1 << 30))])
def test_bad_rotations_are_refused(L, code, change):
    assert _append(L, r=_rope(**change)) == code


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("code,change", [
    (1, dict(q8=None)), (1, dict(mq=None)), (1, dict(kq=None)), (1, dict(seq=None)), (1, dict(pos=None)), (1, dict(o=None)),
    (1, dict(n=0)), (1, dict(max_len=0)), (1, dict(max_len=(1 << 19) + 1)), (1, dict(window=-1)), (1, dict(q8=P + 4)),
    (1, dict(o=P + 4)), (1, dict(stride=8 * 64 - 2)), (1, dict(stride=8 * 64 + 1))])
def test_bad_attention_arguments_are_refused(L, which, code, change):
    assert _attn(L, which, **change) == code


def test_null_structs_are_refused(L):
    n = C.c_longlong(0)
    c = _cache()
    assert L.detint_kv4_workspace(None, 1, 100, C.byref(n)) == 1
    assert L.detint_kv4_workspace(C.addressof(c), 1, 100, None) == 1
    assert L.detint_kv4_append(C.addressof(c), None, P, 768, P, P, 1, P, P, P, None, None, None) == 1


def test_load_kv_refuses_other_widths(L, tiny_artifact):
    h = C.c_void_p()
    for bits in (0, 2, 16, -4):
        assert L.detint_load_kv(tiny_artifact.encode(), 1, 16, bits, None, C.byref(h)) == 1 and not h.value


def test_views_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    import deterministic_integer_only_gb300 as pkg
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        pkg.KV4Cache(u8(4, 2, 64, 32), u8(4, 2, 64, 32), u8(4, 2, 64), u8(4, 2, 64), i32(1, 4), i32(2, 72), 8)
    with pytest.raises(ValueError):
        pkg.RopeNorm(None, None)


@pytest.mark.parametrize("change", [{0: (1 << 27) // 7 + 1}, {2: 1 << 28}, {2: (1 << 31) - 1}, {0: 0}, {2: -3}, {4: 0}, {6: -1},
                                    {1: 0}, {3: 64}, {1: (1 << 31) - 1}, {5: -40}, {5: 90}, {5: (1 << 31) - 1}, {7: 70},
                                    {7: -(1 << 31)}, {8: 4}, {9: -1}, {8 + 31: 1 << 20}])
def test_load_refuses_artifact_scales_outside_the_domain(L, tiny_artifact, tmp_path, change):
    """K/V parameters of the last layer's last kv head that the 4-bit cache's
    arithmetic does not define: refused before anything is sent to a GPU."""
    import hashlib

    import numpy as np

    import float_model
    data = bytearray(open(tiny_artifact, "rb").read())
    kvp = np.array(float_model.load(tiny_artifact)["layers"][-1]["kvp"], np.int32)
    at = data.rfind(kvp.tobytes())
    assert at > 0 and kvp.shape[1] == 40
    for i, x in change.items():
        kvp[-1, i] = x
    data[at:at + kvp.nbytes] = kvp.tobytes()
    path = tmp_path / "changed.detint"
    path.write_bytes(data)
    (tmp_path / "changed.detint.sha256").write_text(hashlib.sha256(data).hexdigest())
    h = C.c_void_p()
    assert L.detint_load_kv(str(path).encode(), 1, 16, 4, None, C.byref(h)) == 5 and not h.value
    assert b"4 bits" in L.detint_last_error()


def test_rotation_tables_and_gammas_in_host_memory_are_refused():
    """The kernels read them: a view of cpu tensors may not reach a launch."""
    torch = pytest.importorskip("torch")
    import deterministic_integer_only_gb300 as pkg
    i16 = lambda *s: torch.zeros(*s, dtype=torch.int16)  # noqa: E731
    with pytest.raises(ValueError, match="cuda"):
        pkg.RopeNorm(i16(16, 32), i16(16, 32))
    with pytest.raises(ValueError, match="cuda"):
        pkg.RopeNorm(None, None, max_pos=16, q_gamma=i16(64), k_gamma=i16(64))
    with pytest.raises(ValueError, match="cuda"):
        pkg.RopeNorm(None, None, max_pos=16, k_gamma=i16(64))


def test_integers_past_32_bits_are_refused(L):
    """They were cut to their low 32 bits on the way to the library: 2^32 + 1
    tokens asked for the workspace of one."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    import deterministic_integer_only_gb300 as pkg
    c = _cache()
    cache = SimpleNamespace(_ref=C.addressof(c), _index=0, device="cuda:0",
                            _torch=SimpleNamespace(_C=SimpleNamespace(_cuda_getDevice=lambda: 0)))
    for n_tok, max_len in (((1 << 32) + 1, 64), (1, (1 << 32) + 64), (1 << 31, 64), (1, -(1 << 32) + 64)):
        with pytest.raises(pkg.DetintError) as e:
            pkg.detint_kv4_workspace(cache, n_tok, max_len)
        assert e.value.code == 1
    for kw in (dict(max_pos=(1 << 32) + 16), dict(max_pos=16, eps=(1 << 32) + 17), dict(max_pos=16, eps=-(1 << 32))):
        with pytest.raises(ValueError):
            pkg.RopeNorm(None, None, **kw)
    assert pkg.RopeNorm(None, None, max_pos=(1 << 31) - 1, eps=17)._c.eps == 17


def test_workspace_query_wants_the_caches_device(L):
    """The split depends on the device's SMs: a query on another current device
    is refused, as the calls it is for are."""
    from types import SimpleNamespace

    import deterministic_integer_only_gb300 as pkg
    c = _cache()
    cache = SimpleNamespace(_ref=C.addressof(c), _index=1, device="cuda:1",
                            _torch=SimpleNamespace(_C=SimpleNamespace(_cuda_getDevice=lambda: 0)))
    with pytest.raises(ValueError, match="current device"):
        pkg.detint_kv4_workspace(cache, 1, 64)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_integers_are_refused(L, off):
    """Int arrays off their natural boundary would be a misaligned access on the
    GPU: an error code on the host instead."""
    n = C.c_longlong(0)
    for name in ("block_table", "status"):
        c = _cache(**{name: P + off})
        assert _append(L, c) == 1 and _attn(L, "decode", c) == 1 and _attn(L, "prefill", c) == 1
        assert L.detint_kv4_workspace(C.addressof(c), 1, 100, C.byref(n)) == 1
    for name in ("seq", "pos", "mq", "kq"):
        assert _append(L, **{name: P + off}) == 1
        assert _attn(L, "decode", **{name: P + off}) == 1 and _attn(L, "prefill", **{name: P + off}) == 1
        assert b"aligned" in L.detint_last_error()
