"""mx_kv_accept_fp4's C ABI without layers, on the host with no GPU: its arguments are looked at where new lengths are
wanted; without them, or without caches, the call does nothing."""
import ctypes

import pytest

import block_scaled_precision_act_amd as mx
from test_draft_abi import ACCEPT, A, AL, B, N, OK, S, ST, _call, _expect, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("change,status", [
    ({}, "device"), (dict(q_starts=A, max_q=64), "device"), (dict(width=0, path=0), "device"), (dict(lens_out=0), OK),
    (dict(lens_out=0, seq_lens=0), OK), (dict(batch=0, total_q=0), OK), (dict(seq_lens=0), N), (dict(count=0), N),
    (dict(path=0), N), (dict(lens_out=B + 2), AL), (dict(count=A + 2), AL), (dict(lens_out=A), ST), (dict(max_q=6), S),
    (dict(layers=-1), S), (dict(width=-1), S), (dict(batch=65536, total_q=5 * 65536), S)])
def test_accept_without_layers(lib, change, status):  # noqa: F811
    nothing = ctypes.create_string_buffer(1)
    expected = _expect(status)
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "layers": 0, "caches": ctypes.addressof(nothing)}, change) == expected


def test_accept_without_layers_or_caches_does_nothing(lib):  # noqa: F811
    assert _call(lib, "mx_kv_accept_fp4", {**ACCEPT, "layers": 0, "caches": 0}, {}) == mx.MX_OK
