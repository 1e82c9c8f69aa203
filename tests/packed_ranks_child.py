"""Run by test_gpu_zz_packed_ranks.py in a fresh process (NCCL lives only there).

A packed step whose targets are counted and whose gradients are averaged over a one-rank
communicator, on a plain and on a sharded stack, must be the plain packed step bit for bit.
"""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]


def main():
    import torch
    from layer_streamed_qlora_nf4_b200 import lib as L
    from layer_streamed_qlora_nf4_b200 import synth
    from test_gpu_packed_step import _batch, _optimiser, _run
    from test_gpu_stack import Stack
    L.load()
    st = Stack(L, synth.SMALL, 5)
    runs = []
    for form in ("plain", "reduced", "sharded and reduced"):
        if form.startswith("sharded"):
            S = L.lsq_shard_bytes(st.blob_bytes, 1)
            bufs = [torch.empty(S, dtype=torch.uint8, device="cuda") for _ in range(2)]
            h = L.StreamStack(st.cfg, st.host_blobs, bufs[0], bufs[1], False)
            h.shard(L.lsq_nccl_unique_id(), 1, 0, S)
        else:
            h = st.handle(L, resident=False)
        if form != "plain":
            h.reduce_grads(L.lsq_nccl_unique_id(), 1, 0)
        lora = st.lora.clone()
        grad = torch.full_like(lora, float("nan"))
        opt, parts = _optimiser(L, st.cfg, lora, grad)
        kept = []
        for step in (1, 2, 3):
            d = _batch(40 + step, step == 2, step > 1)[2]
            if step == 3:
                d["loss_mask"].zero_()            # a rank without targets
            loss, logits, _, _ = _run(L, st, h, d, opt=opt, step=step, lora=lora, grad=grad)
            assert (loss == 0.0) == (step == 3)
            kept += [torch.tensor(loss), logits.clone(), grad.clone(), lora.clone()]
        runs.append(kept + [t.clone() for k in (2, 3, 4, 5) for t in parts[k]])
        h.close()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
    assert L.lsq_device_status() == 0
    print("packed ranks ok")


if __name__ == "__main__":
    main()
