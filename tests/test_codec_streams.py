"""Where the codec's tensor forms take their memory when they are given a
stream of their own, shown on the host with stand-ins for the streams and the
library."""
import pytest
import torch

import lossless_compression_float_amd as uz
from test_linear_streams import Library, streams  # noqa: F401  (a fixture)

T = torch.zeros(100, dtype=torch.bfloat16)
FRAME = torch.zeros(300, dtype=torch.uint8)

CALLS = {
    "compress": lambda **kw: uz.compress(T, **kw),
    "decompress": lambda **kw: uz.decompress(FRAME, torch.bfloat16, 100, **kw),
    "compress_arbitrated": lambda **kw: uz.compress_arbitrated(T, uz.policy(), **kw),
    "compress_batched": lambda **kw: uz.compress_batched([T, T], **kw),
    "decompress_batched": lambda **kw: uz.decompress_batched([FRAME], torch.bfloat16, [100], **kw),
    "compress_batched_arbitrated": lambda **kw: uz.compress_batched_arbitrated([T], uz.policy(), **kw),
}


class Codec(Library):
    def __getattr__(self, name):
        fn = super().__getattr__(name)
        return (lambda *a: 1000) if "_size" in name else fn


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_another_stream_takes_its_memory_there(streams, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(uz, "lib", Codec)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    main, side = streams["main"], streams["side"]
    results = CALLS[name](stream=side)
    assert len(streams["made"]) >= 3 and all(s is side for _, s in streams["made"]), streams["made"]
    for r in results:
        for t in [r] if isinstance(r, torch.Tensor) else r:
            assert main in [s for p, s in streams["recorded"] if p == t.data_ptr()]
    assert streams["current"] is main


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_the_current_stream_records_nothing(streams, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(uz, "lib", Codec)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    CALLS[name]()
    CALLS[name](stream=streams["main"])
    assert all(s is streams["main"] for _, s in streams["made"]) and not streams["recorded"]
