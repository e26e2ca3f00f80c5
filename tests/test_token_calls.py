"""The binding's marshalling of the single-token calls: what reaches the C entry,
and what is refused, on host tensors and with recorders in place of the C
entries (no GPU, no launch)."""
import ctypes

import numpy as np
import pytest
import torch

import block_causal_attention_wave_b200 as wave
from block_causal_attention_wave_b200 import _binding

P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
NAMES = ("wave_linear_bias", "wave_rotary", "wave_kv_write_tokens", "wave_token_attn")
HOST = -1  # a host tensor's get_device()


@pytest.fixture()
def calls():
    """(module, record): the module bound to recorders; record holds the last call."""
    wave.load()
    module = pytest.importorskip("block_causal_attention_wave_b200._call")
    record = {}

    def recorder(name):
        types = _binding._SIGS[name][1]

        def fn(*args):
            record.update(name=name, args=args, rc=0)
            if name == "wave_kv_write_tokens":  # the arrays live as long as the call
                n = args[1]
                record["nodes"] = ctypes.string_at(args[2], 8 * n)
                record["first"], record["counts"] = (ctypes.string_at(args[i], 4 * n) for i in (3, 4))
            if name == "wave_token_attn":
                n = args[2]
                record["nodes"] = ctypes.string_at(args[1], 8 * n)
                record["own"] = ctypes.string_at(args[4], 4 * n) if args[4] else None
            return -7 if record.get("fail") else 0
        plain = [P if t is ctypes.c_char_p or not isinstance(t(), ctypes._SimpleCData) else t for t in types]
        return ctypes.CFUNCTYPE(ctypes.c_int, *plain)(fn)
    keep = [recorder(n) for n in NAMES]
    module.bind(*(ctypes.cast(f, P).value for f in keep), torch.bfloat16, torch.float32, torch.int32)
    yield module, record
    _binding._call = None  # the next call of a cache binds the library again


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def ints(b):
    return np.frombuffer(b, np.int32).tolist()


def test_linear_arguments(calls):
    m, rec = calls
    A, W, b = z(3, 80)[:, :64], z(8, 64), z(8)
    Y, R = z(3, 40)[:, 8:16], z(3, 16)[:, :8]
    assert m.linear_bias(77, HOST, A, W, Y, b, R, 2, 99) == 0
    assert rec["args"] == (77, A.data_ptr(), 80, 3, 64, W.data_ptr(), 8, b.data_ptr(), R.data_ptr(), 16, 2,
                           Y.data_ptr(), 40, 99)
    m.linear_bias(77, HOST, z(1, 80)[:, :64], W, z(1, 8), None, None, 0, 0)
    a = rec["args"]
    assert a[2:5] == (64, 1, 64) and a[7] is None and a[8] is None and a[9] == 0 and a[-1] is None
    # heads side by side are one row; a bias of any shape that holds N values in order
    m.linear_bias(77, HOST, z(3, 64), W, z(3, 2, 4), b.view(1, 8), None, 0, 0)
    assert rec["args"][12] == 8
    rec["fail"] = True
    assert m.linear_bias(77, HOST, A, W, Y, None, None, 0, 0) == -7
    assert m.linear_bias(None, HOST, A, W, Y, None, None, 0, 0) == -7 and rec["args"][0] is None


def test_rotary_arguments(calls):
    m, rec = calls
    spec = _binding.RotarySpec((1, 2, 3), 10.0, 0, 1, 0)
    pos, wide = z(5, 3, dtype=torch.int32), z(5, 9 * 64 + 8)
    Q, K = wide[:, :256].unflatten(1, (4, 64)), \
        wide[:, 256:384].unflatten(1, (2, 64))
    out = z(5, 4, 64)
    assert m.rotary(7, HOST, 64, ctypes.addressof(spec), pos, Q, K, out, K, 0) == 0
    a = rec["args"]
    assert a[2:] == (pos.data_ptr(), 5, Q.data_ptr(), 584, 4, out.data_ptr(), 256, K.data_ptr(), 584, 2,
                     K.data_ptr(), 584, None)
    m.rotary(7, HOST, 64, ctypes.addressof(spec), pos, Q, None, Q, None, 3)
    assert rec["args"][9:] == (None, 0, 0, None, 0, 3)


def test_write_arguments(calls):
    m, rec = calls
    kv = z(6, 2, 2, 64)
    K, V = kv[:, 0], kv[:, 1]
    assert m.write_tokens(7, HOST, 128, [(0, 1), (np.int32(5), 2)], [9, np.int64(8)], [4, 2], K, V, 0) == 0
    assert rec["args"][1] == 2 and rec["args"][5:] == (K.data_ptr(), 256, V.data_ptr(), 256, None)
    assert ints(rec["nodes"]) == [0, 1, 5, 2] and ints(rec["first"]) == [9, 8] and ints(rec["counts"]) == [4, 2]
    m.write_tokens(7, HOST, 128, ((-1, 0), (3, 1)), (0, 5), None, K[:2], V[:2], 0)
    assert ints(rec["nodes"]) == [-1, 0, 3, 1] and ints(rec["counts"]) == [1, 1]
    assert m.write_tokens(7, HOST, 128, [], [], [], K[:0], V[:0], 0) == 0 and rec["args"][1] == 0


def test_attention_arguments(calls):
    m, rec = calls
    Q, O, lse, ws = z(2, 6, 64), z(2, 400)[:, :384], z(2, 6, dtype=torch.float32), z(100, dtype=torch.float32)
    assert m.token_attn(7, HOST, 64, [(1, 2), (3, 4)], 1, Q, O, [5, 0], lse, ws, 9) == 0
    a = rec["args"]
    assert a[2:4] == (2, 1) and a[5:] == (6, Q.data_ptr(), 384, O.data_ptr(), 400, lse.data_ptr(),
                                           ws.data_ptr(), 400, 9)
    assert ints(rec["nodes"]) == [1, 2, 3, 4] and ints(rec["own"]) == [5, 0]
    m.token_attn(7, HOST, 64, [(1, 2), (3, 4)], 1, Q, O, None, None, None, 0)
    assert rec["own"] is None and rec["args"][10:13] == (None, None, 0)


def test_refusals(calls):
    m, rec = calls
    W, q, pos, h = z(8, 64), z(3, 2, 64), z(3, 3, dtype=torch.int32), z(2, 2, 64)
    spec = ctypes.addressof(_binding.RotarySpec((1, 2, 3), 10.0, 0, 1, 0))
    lin = lambda *a: m.linear_bias(7, HOST, *a)  # noqa: E731
    rot = lambda *a: m.rotary(7, HOST, 64, spec, *a, 0)  # noqa: E731
    wr = lambda *a: m.write_tokens(7, HOST, 128, *a, 0)  # noqa: E731
    at = lambda *a: m.token_attn(7, HOST, 64, *a, 0)  # noqa: E731
    one = [(0, 1)]
    bad = [
        lambda: m.linear_bias(7, 0, z(3, 64), W, z(3, 8), None, None, 0, 0),        # another device
        lambda: lin(z(3, 64, dtype=torch.float16), W, z(3, 8), None, None, 0, 0),
        lambda: lin(z(2, 3, 64), W, z(3, 8), None, None, 0, 0),
        lambda: lin(z(3, 64), z(8, 72), z(3, 8), None, None, 0, 0),
        lambda: lin(z(3, 64), z(8, 128)[:, :64], z(3, 8), None, None, 0, 0),
        lambda: lin(z(64, 3).t(), W, z(3, 8), None, None, 0, 0),
        lambda: lin(z(3, 64), W, z(2, 8), None, None, 0, 0),
        lambda: lin(z(3, 64), W, z(3, 4, 8)[:, :, :2], None, None, 0, 0),           # heads with gaps
        lambda: lin(z(3, 64), W, z(1, 1, 1, 3, 8), None, None, 0, 0),
        lambda: lin(z(3, 64), W, z(3, 8), z(7), None, 0, 0),
        lambda: lin(z(3, 64), W, z(3, 8), z(16)[::2], None, 0, 0),
        lambda: lin(z(3, 64), W, z(3, 8), z(8, dtype=torch.float32), None, 0, 0),
        lambda: lin(z(3, 64), W, z(3, 8), None, z(3, 16), 0, 0),
        lambda: rot(z(3, 3, dtype=torch.int64), q, None, q, None),
        lambda: rot(z(2, 3, dtype=torch.int32), q, None, q, None),
        lambda: rot(z(3, 4, dtype=torch.int32)[:, :3], q, None, q, None),
        lambda: rot(pos, z(3, 2, 32), None, q, None),
        lambda: rot(pos, q, None, z(2, 2, 64), None),
        lambda: rot(pos, q, z(2, 2, 64), q, z(2, 2, 64)),
        lambda: rot(pos, z(3, 64, 2).transpose(1, 2), None, q, None),
        lambda: wr(one, [0], None, h, h[:1]),
        lambda: wr(one, [0, 1], None, h[:1], h[:1]),
        lambda: wr(one, [0], [1, 1], h, h),
        lambda: wr(one, [0], [-1], h[:1], h[:1]),
        lambda: wr([(0, 1, 2)], [0], None, h[:1], h[:1]),
        lambda: wr([(0,), (0, 1, 2)], [0, 0], None, h, h),
        lambda: at(one, 1, q, h[:1], None, None, None),
        lambda: at(one, 1, h[:1], h[:1], [1, 2], None, None),
        lambda: at(one, 1, h[:1], h[:1], None, z(1, 2), None),
        lambda: at(one, 1, h[:1], h[:1], None, None, z(9, 9).t()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call, error in [
        (lambda: lin(z(3, 64), W, z(3, 8), None, None, 0), TypeError),               # an argument short
        (lambda: lin(None, W, z(3, 8), None, None, 0, 0), AttributeError),
        (lambda: lin(z(3, 64), W, None, None, None, 0, 0), AttributeError),
        (lambda: rot(None, q, None, q, None), AttributeError),
        (lambda: rot(pos, q, q, q, None), AttributeError),
        (lambda: wr(5, [0], None, h, h), TypeError),
        (lambda: wr([5], [0], None, h, h), TypeError),
        (lambda: wr([(0, 1 << 40)], [0], None, h, h), OverflowError),
        (lambda: wr(one, [1 << 31], None, h, h), OverflowError),
        (lambda: wr(one, [0.5], None, h, h), TypeError),
        (lambda: at(one, 1, h[:1], h[:1], 5, None, None), TypeError),
    ]:
        with pytest.raises(error):
            call()
    assert "args" not in rec, "nothing reached a C entry"
