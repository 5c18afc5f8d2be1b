"""Calls on a stream that is not torch's current one (the ``stream`` argument
of the torch calls: a stream's handle, as ``torch.cuda.Stream.cuda_stream``)
that allocate their outputs."""
from __future__ import annotations


def elsewhere(call, stream, *args, **kw):
    """``call(*args, **kw)``, which works on the current stream, on the stream
    of handle ``stream`` instead.

    What the call allocates comes from that stream's memory: a block that the
    current stream has given back may still be in use there.  Its results are
    used on the current stream next, so their memory is kept, after they are
    dropped, until that stream's work so far is done.  Operands are the
    caller's to keep until the call's work is done."""
    import torch
    operands = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor) and t.is_cuda]
    if not operands:
        return call(*args, **kw)    # which says what is wrong
    device = operands[0].device
    now = torch.cuda.current_stream(device)
    if stream == now.cuda_stream:
        return call(*args, **kw)
    # 0 and 1 both name the legacy default stream.
    there = torch.cuda.default_stream(device) if stream in (0, 1) else \
        torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(there):
        results = call(*args, **kw)
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None and not any(t is o for o in operands):
            t.record_stream(now)
    return results
