// A paged latent cache: one vector of a latent part and a rotated key part for every slot.
#pragma once

#include "fa_lm.cuh"

// checks a latent cache's description and makes the kernels' view of it: rows of one head
inline fa_status fa_view_latent(const char *fn, const fa_latent_cache *c, const int32_t *page_table, int32_t max_pages,
                                fa_cache_view *out) {
    if (!c) return fa_refuse(fn, "NULL cache");
    if (c->format != FA_CACHE_F16 && c->format != FA_CACHE_BF16) return fa_refuse(fn, "a latent cache is fp16 or bf16");
    if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fa_refuse(fn, "page_size must be a power of two in [1, 1024]");
    if (c->n_pages < 0 || (int64_t)c->n_pages * c->page_size > 2147483647) return fa_refuse(fn, "n_pages * page_size out of range");
    if (c->latent_dim < 128 || c->latent_dim > 512 || c->latent_dim % 128)
        return fa_refuse(fn, "latent_dim must be a multiple of 128 in [128, 512]");
    if (c->rope_dim < 16 || c->rope_dim > 64 || c->rope_dim % 16)
        return fa_refuse(fn, "rope_dim must be a multiple of 16 in [16, 64]");
    if (max_pages < 0) return fa_refuse(fn, "max_pages < 0");
    if (c->n_pages > 0 && !c->rows) return fa_refuse(fn, "NULL cache buffer");
    if ((uintptr_t)c->rows & 15) return fa_refuse(fn, "cache rows must be 16-byte aligned");
    if (max_pages > 0 && !page_table) return fa_refuse(fn, "NULL page_table");
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    *out = fa_cache_view{c->rows, nullptr, nullptr, nullptr, c->n_pages, shift, 1, c->latent_dim + c->rope_dim, page_table, max_pages};
    return FA_OK;
}
