// zero1_adamw_plan.h -- host-only rules of AdamW over a list of tensors
// (zero1_adamw.cu): the norm's launches and the partial sums they write, and
// which buffers of a step share memory.
// Plain C++, so that the rules are tested without a GPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace zero1 {

constexpr uint32_t kListBlock = 256;      // entries of one block: 8 a lane of one warp
constexpr int kListThreads = 256;
constexpr uint32_t kWarps = kListThreads / 32;
constexpr uint32_t kNormBlocks = 8;       // blocks of a warp of the norm, at a time (4: 68 us in place of 63, 2: 68 to 80)

// Tensors whose pointers one launch holds: kernel arguments are 32,764 bytes
// at most, and longer ones take longer to launch.
constexpr int kCaps[3] = {32, 256, 1600};

// Thread blocks of the norm's launch over `nblocks` blocks of the list, each
// of which writes one partial sum: the four an SM that run at once, or one for
// each 64 blocks.  The step's last launch forms the norm, and so has one even
// where its tensors are all empty; another launch without blocks is left out (0).
inline uint32_t norm_grid(uint64_t nblocks, bool last, int sms)
{
    const uint64_t need = (nblocks + kWarps * kNormBlocks - 1) / (kWarps * kNormBlocks);
    const uint32_t grid = (uint32_t)std::min<uint64_t>(need, 4ull * (uint64_t)sms);
    return grid == 0 && last ? 1 : grid;
}

// Partial sums of a step whose launches take `cap` tensors each; tensor i has
// the blocks first[i] to first[i + 1].
inline uint64_t norm_partials(const uint64_t *first, uint64_t count, uint64_t cap, int sms)
{
    uint64_t n = 0;
    for (uint64_t i = 0; i < count; i += cap) {
        const uint64_t end = std::min(i + cap, count);
        n += norm_grid(first[end] - first[i], end == count, sms);
    }
    return n;
}

// A buffer of the state: where it begins, its bytes.
struct StateBuffer {
    const void *p;
    uint64_t bytes;
};

// A step's tensors (sizes[i] entries each) and the bytes of an entry.
struct ListTensors {
    const uint64_t *sizes;
    size_t count;
    const void *const *grads;
    void *const *params;
    uint64_t grad_bytes, param_bytes;
};

// The first tensor of which the parameter or the gradient shares memory with
// a buffer of the state (count: none does), and that buffer's number.
inline size_t tensor_in_state(const ListTensors &t, const StateBuffer *state, int buffers, int *which, bool *param)
{
    for (size_t i = 0; i < t.count; ++i) {
        if (t.sizes[i] == 0) continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(t.params[i]), p_end = p + t.sizes[i] * t.param_bytes;
        const uintptr_t g = reinterpret_cast<uintptr_t>(t.grads[i]), g_end = g + t.sizes[i] * t.grad_bytes;
        for (int k = 0; k < buffers; ++k) {
            if (!state[k].p) continue;
            const uintptr_t from = reinterpret_cast<uintptr_t>(state[k].p), to = from + state[k].bytes;
            *param = p < to && from < p_end;
            if (!*param && !(g < to && from < g_end)) continue;
            *which = k;
            return i;
        }
    }
    return t.count;
}

// A tensor's bytes, for shared_param.
struct TensorRange {
    uintptr_t from, to;
    size_t tensor;
    bool param;
};

// A parameter tensor that shares memory with another tensor of the call
// (count: there is none): each is written by blocks that run in any order.
// `ranges` is room for 2 count of them; nothing is allocated.
inline size_t shared_param(const ListTensors &t, TensorRange *ranges)
{
    // parameters in the order of their addresses, gradients all before or all after them: nothing to sort
    uintptr_t p_end = 0, p_begin = UINTPTR_MAX, g_begin = UINTPTR_MAX, g_end = 0;
    bool ordered = true;
    size_t n = 0;
    for (size_t i = 0; i < t.count; ++i) {
        if (t.sizes[i] == 0) continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(t.params[i]), g = reinterpret_cast<uintptr_t>(t.grads[i]);
        const uintptr_t p_to = p + t.sizes[i] * t.param_bytes, g_to = g + t.sizes[i] * t.grad_bytes;
        ordered = ordered && p >= p_end;
        p_begin = std::min(p_begin, p);
        p_end = std::max(p_end, p_to);
        g_begin = std::min(g_begin, g);
        g_end = std::max(g_end, g_to);
        ranges[n++] = {p, p_to, i, true};
        ranges[n++] = {g, g_to, i, false};
    }
    if (ordered && (g_end <= p_begin || p_end <= g_begin)) return t.count;
    std::sort(ranges, ranges + n, [](const TensorRange &a, const TensorRange &b) { return a.from < b.from; });
    // the furthest end so far, of parameters and of anything
    const TensorRange *any = nullptr, *param = nullptr;
    for (const TensorRange *r = ranges; r != ranges + n; ++r) {
        if ((r->param && any && any->to > r->from) || (param && param->to > r->from)) return r->param ? r->tensor : param->tensor;
        if (!any || r->to > any->to) any = r;
        if (r->param && (!param || r->to > param->to)) param = r;
    }
    return t.count;
}

}  // namespace zero1
