// Whole-number arithmetic of the adapters' outer products: how the tokens of an
// adapter are counted, cut into parts and found again.  Plain functions for the
// device and the host, so that a host program can run them on index arrays that
// no kernel should be tried on.
//
// Offsets come from device memory and nothing can check them on the host.  In
// order, the segments of an adapter hold at most M tokens together; out of order
// they can hold 2^31 times that.  So every count is capped at M, and then no sum
// leaves 32 bits, whatever the arrays hold, and in ordered arrays no cap is met.
#pragma once

#ifdef __HIP__
#define SS1_LIST_FN __host__ __device__ __forceinline__
#else
#define SS1_LIST_FN inline
#endif

namespace ss1 {

// a + b, at most `most`; a and b in [0, most].
SS1_LIST_FN int add_capped(int a, int b, int most) {
    const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
    return s < static_cast<unsigned>(most) ? static_cast<int>(s) : most;
}

// Where a segment's tokens stand in the list of its adapter's: places [first,
// end), and the token at a place is start + place.
struct ListRun {
    int end, start;
};

// A segment from token b on, of n tokens, with `first` tokens of the adapter
// before it.
SS1_LIST_FN ListRun list_run(int b, int n, int first, int M) { return {add_capped(first, n, M), b - first}; }

// Parts of P tokens that an adapter's tokens are cut into, and the end of part i.
SS1_LIST_FN int parts_of(int tokens, int P) { return tokens > P ? (tokens - 1) / P + 1 : 1; }
SS1_LIST_FN int part_end(int tokens, int P, int i) { return tokens - i * P > P ? (i + 1) * P : tokens; }

// Entries, slots and adapters with several parts so far, and the adapter's own
// place after them; sums that passed their array stay there, past its end.
struct PlanSums {
    int entries, slots, several;
};
SS1_LIST_FN PlanSums plan_add(PlanSums a, PlanSums b, int most, int slots) {
    return {a.entries + b.entries < most ? a.entries + b.entries : most,
            a.slots + b.slots < slots ? a.slots + b.slots : slots, a.several + b.several};
}

}  // namespace ss1
