"""Helpers of the cache tests: NumPy caches to the GPU and back."""
import numpy as np

from gpu_helpers import torch_mod


def up(a, dtype=None):
    torch = torch_mod()
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype=dtype))).to("cuda:0")


def upload_cache(c):
    import bit_quantized_decode_qmv_amd as bq
    return bq.KVCache(up(c["k"]), up(c["v"]), up(c["ks"], np.float32), up(c["vs"], np.float32), c["format"])


def download_cache(cache):
    return {"k": cache.k.cpu().numpy(), "v": cache.v.cpu().numpy(), "ks": cache.k_scales.cpu().numpy(),
            "vs": cache.v_scales.cpu().numpy(), "format": cache.format}


def cu_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
