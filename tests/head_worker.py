"""Worker of tests/test_gpu_head_builds.py, run in a subprocess (the library and LORA_PDL are read
once per process): forwards and backwards of the LM head's operators on ragged shapes, printing one
JSON line with the library loaded, a SHA-256 of every output's bits per case and the device status."""
import hashlib
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# rows, width, vocabulary, tokens, alternatives: few rows (one range, several tiles a range), the
# pair kernels with ragged rows, columns and widths, splits and one piece, compacted rows
CASES = [(3, 200, 1000, 1, 5), (100, 72, 30000, 3, 32), (129, 72, 520, 3, 7), (700, 200, 2056, 5, 0),
         (2600, 1032, 1000, 2, 4)]


def main():
    import torch

    import qlora_linear_b200 as q
    from synth import HeadCase, make_head_case
    from tests.gpu_helpers import dev_bf16

    res = {"lib": os.path.basename(q.LIB_PATH), "cases": {}, "status": []}
    for case in CASES:
        M, D, V, n, k = case
        inp = make_head_case(HeadCase("worker", M, D, V, n, 7000 + M, ignore_frac=0.3))
        W = q.LoraWeight.bf16(dev_bf16(inp["W"]))
        x = dev_bf16(inp["X"])
        ids, t, dl, dlp, dent = (torch.from_numpy(inp[a]).cuda()
                                 for a in ("ids", "teacher", "dloss", "dlogprob", "dentropy"))
        h = hashlib.sha256()
        for slice_ in (0, 512):
            lp, kd = q.LoraTokenLogProbs(W, slice_=slice_), q.LoraDistill(W, slice_=slice_)
            for save in (False, True):
                o = lp.forward(x, ids, top_k=k, save=save)
                d = kd.forward(x, ids, t, save=save)
                outs = [o.logprob, o.entropy, o.lse, d.loss, lp.backward(x, ids, o, dlp, dent),
                        kd.backward(x, ids, t, d, dl)]
                if k:
                    outs += [o.top_ids, o.top_logprob]
                for a in outs:
                    h.update(a.contiguous().view(torch.uint8).cpu().numpy().tobytes())
            res["status"] += [lp.status(), kd.status()]
        res["cases"][str(case)] = h.hexdigest()
    print(json.dumps(res), flush=True)


if __name__ == "__main__":
    main()
